"""The example's speculative step with 8-bit decoder layers, call by call: each
operator's outputs are within the counted roundings of its definition in 64
bits on the very inputs that the step gave it (the codes, which other
operators' roundings may move, bit for bit on theirs)."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R
import tree_ref as T
from test_gpu_int8_step import E

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _raw(t):
    return t.cpu().numpy()


def _held(got, want, bound):
    worst = (np.abs(_np(got) - want) / bound).max()
    assert worst <= 1.0, worst


class Calls:
    """The calls of the decoder-layer operators, with copies of their inputs
    and outputs, checked one by one."""
    NAMES = ("residual_norm", "gemm_w8a8", "gated_w8a8", "quant_rows_int8", "rotate", "tree_attention")

    def __init__(self, monkeypatch):
        self.seen = []
        for name in self.NAMES:
            monkeypatch.setattr(vq, name, self._wrapped(name, getattr(vq, name)))

    def _wrapped(self, name, fn):
        def copy(v):
            return v.clone() if isinstance(v, torch.Tensor) else v

        def call(*args, **kw):
            before = [copy(a) for a in args], {k: copy(v) for k, v in kw.items()}
            got = fn(*args, **kw)
            after = {k: copy(v) for k, v in kw.items()}
            self.seen.append((name, *before, copy(got) if isinstance(got, torch.Tensor) else [copy(g) for g in got], after))
            return got
        return call

    def check(self):
        for name, args, kw, got, after in self.seen:
            getattr(self, name)(args, kw, got, after)

    def residual_norm(self, args, kw, got, after):
        x, y, w = args
        want, ex, h, eh = R.norm(_np(x), _np(y), _np(w), None, None, 1.0, float(np.float32(1e-6)))
        if y is not None:
            _held(after["residual_out"], want, R.rounded(want, ex, "f32"))
        q, s = _np(got[0]), _np(got[1])
        top, at = np.abs(h).max(1), np.abs(h).argmax(1)
        # the scale: the error of whichever element is the largest, and its division
        assert (np.abs(s * 127 - top) <= eh.max(1) + 2 * R.U * top + eh[np.arange(len(h)), at]).all()
        # a code: half a step, what its element is off, and the quotient's rounding of at most 127 steps
        assert (np.abs(q * s[:, None] - h) <= 0.5 * s[:, None] + eh + 127 * 2 * R.U * s[:, None]).all()

    def quant_rows_int8(self, args, kw, got, after):
        q, s = R.quant(args[0].float().cpu().numpy())
        assert np.array_equal(_raw(got[0]), q) and np.array_equal(_raw(got[1]), s)

    def gemm_w8a8(self, args, kw, got, after):
        w, ws, x, xs = (_raw(t) for t in args[:4])
        y, err = R.product(x, xs, w, ws)
        _held(got, y, R.rounded(y, err, "bf16"))

    def gated_w8a8(self, args, kw, got, after):
        wg, gs, wu, us, x, xs = (_raw(t) for t in args[:6])
        y, err = R.gated(x, xs, wg, gs, wu, us, "silu")
        _held(got, y, R.rounded(y, err, "bf16"))

    @staticmethod
    def _masks(kw):
        m = kw.get("tree_mask")
        return None if m is None else _raw(m).view(np.uint64)

    def rotate(self, args, kw, got, after):
        q, k, freq, lens = args
        pos = R.positions(_raw(lens), self._masks(kw), q.shape[1])
        for out, t in zip(got, (q, k)):
            y, err = R.rotate(_np(t), pos, _raw(freq), False, 1.0)
            _held(out, y, R.rounded(y, err, "bf16"))

    def tree_attention(self, args, kw, got, after):
        q, k, v, kc, vc, table, lens = args
        y, bound = T.attention(_np(q), _np(k), _np(v), _np(kc), _np(vc), _raw(table), _raw(lens), self._masks(kw), None,
                               q.shape[-1] ** -0.5, "bf16")
        _held(got, y, bound)


@pytest.mark.parametrize("nodes,kind", [(12, "tree"), (5, "chain"), (1, "chain")])
def test_every_call_of_a_step(monkeypatch, nodes, kind):
    B, prompt_len = 3, 37
    model = E.Int8Model(seed=4)
    g = torch.Generator(device=model.device)
    g.manual_seed(9)
    prompt = torch.randint(0, model.vocab, (B, prompt_len), generator=g, device=model.device, dtype=torch.int32)
    cache = E.Cache(model, B, prompt_len + 3 * nodes)
    calls = Calls(monkeypatch)
    _, keys, values = model.forward(prompt[:, :-1].contiguous(), cache)  # a prompt, nothing cached
    per = 10 * model.layers + 2  # ten a layer, the last norm and the head
    assert len(calls.seen) == per
    calls.check()
    cache.append(keys, values)
    tree = E.Tree([-1] + [(i - 1) // 3 if kind == "tree" else i - 1 for i in range(1, nodes)], B, model.device)
    root = prompt[:, -1]
    for _ in range(2):  # over the cache, at ragged lengths from the second step on
        calls.seen.clear()
        out, count = E.step(model, cache, tree, root, g)
        assert len(calls.seen) == per
        calls.check()
        root = out.gather(1, (count.long() - 1)[:, None])[:, 0]
