"""The cached workspace of the speculative-step operators under host threads
and under graphs."""
import threading

import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
from test_gpu_tree_attention import Case
from test_gpu_tree_verify import _dev, _inputs, _run

pytestmark = pytest.mark.gpu


def _attention_call(seed):
    c = Case(seed, "bf16", 8, 8, 2, 128, 64, [3000, 500], mask="tree")
    dev = [t.cuda() for t in (c.q, c.k, c.v, c.k_cache, c.v_cache, torch.from_numpy(c.table), torch.from_numpy(c.lens))]
    masks = torch.from_numpy(c.masks.view(np.int64)).cuda()
    return lambda: vq.tree_attention(*dev, tree_mask=masks, scale=c.scale)


def _verify_call(seed):
    dev = {k: _dev(x) for k, x in _inputs(seed, 7, 16, 20001, "bf16", True).items()}
    return lambda: torch.cat([t.view(-1) for t in vq.tree_verify(
        dev["target"], dev["draft"], dev["tokens"], dev["uniforms"], dev["noise"], parents=dev["parents"],
        temperature=dev["temperature"])])


def _greedy_call(seed):
    g = torch.Generator().manual_seed(seed)
    logits, draft = torch.randn(16, 50000, generator=g).cuda(), torch.zeros(15, dtype=torch.int32, device="cuda")
    return lambda: torch.cat(vq.greedy_verify(logits, draft))


@pytest.mark.parametrize("make", [_attention_call, _verify_call, _greedy_call])
def test_two_threads_on_one_stream(make):
    """Two host threads, the same stream, the default workspace: each gets its
    own results every time."""
    calls = [make(950), make(951)]
    want = [c().cpu() for c in calls]
    got = [[], []]

    def work(i):
        for _ in range(100):
            got[i].append(calls[i]())
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 100 and all(torch.equal(x.cpu(), want[i]) for x in got[i])


def test_graph_keeps_its_cached_workspace():
    """A graph captured with the default workspace, which a larger call on the
    same stream then replaces: replays give the same results and write to
    nothing allocated since."""
    c = _inputs(960, 7, 16, 20001, "bf16", True)
    want = _run(c)
    dev = {k: _dev(x) for k, x in c.items()}
    big = {k: _dev(x) for k, x in _inputs(961, 30, 16, 20001, "bf16", True).items()}
    outs = [torch.empty(7, 16, dtype=torch.int32, device="cuda") for _ in range(2)] + \
        [torch.empty(7, dtype=torch.int32, device="cuda")]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(d, **kw):
        return vq.tree_verify(d["target"], d["draft"], d["tokens"], d["uniforms"], d["noise"], parents=d["parents"],
                              temperature=d["temperature"], **kw)
    small = vq.tree_verify_workspace_bytes(7, 16, 20001)
    with torch.cuda.stream(s):
        call(dev)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(dev, tokens_out=outs[0], path_out=outs[1], count_out=outs[2])
    with torch.cuda.stream(s):
        call(big)
        s.synchronize()
        filled = [torch.full((small,), 0x3C, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs:
            o.fill_(-9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert np.array_equal(x.cpu().numpy(), y)
        assert all(bool((t == 0x3C).all()) for t in filled)
