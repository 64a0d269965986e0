"""The binding's cached workspaces on the host: a stand-in for the library
records which buffer each call was given and when."""
import gc
import threading
import time
import weakref

import pytest
import torch

import block_quantized_gemm_amd as vq

STREAM = 7


class Stream:
    cuda_stream = STREAM

    def synchronize(self):
        pass


class Lib:
    """Answers workspace queries with `need` bytes and notes the calls: a call
    stays inside for a while, or until a second one has joined it."""

    def __init__(self, need=1024):
        self.need, self.guard, self.inside, self.shared = need, threading.Lock(), [], False
        self.joined, self.seen = threading.Event(), []

    def _call(self, workspace):
        with self.guard:
            self.seen.append(workspace)
            self.shared = self.shared or workspace in self.inside
            self.inside.append(workspace)
            if len(self.inside) > 1:
                self.joined.set()
        self.joined.wait(self.patience)
        with self.guard:
            self.inside.remove(workspace)
        return vq.VQ_OK

    patience = 0.0

    def __getattr__(self, name):
        if "workspace_bytes" in name:
            return lambda *sizes: self.need
        return lambda *args: self._call(args[-3])  # workspace, bytes, stream end every list


@pytest.fixture
def fake(monkeypatch):
    """The binding on host tensors: no device, one stream, the stand-in library."""
    lib = Lib()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name, value in (("lib", lambda: lib), ("_stream", lambda s: STREAM), ("_raw_stream", lambda s: STREAM),
                        ("_auto_ws", {}), ("_ws_needs", {}), ("_dev_ptr", lambda t, name: t.data_ptr()),
                        ("_array", lambda t, name, shape, dtype: None if t is None else t.data_ptr()),
                        ("_rows", lambda t, name, shape: shape[-2] * shape[-1])):
        monkeypatch.setattr(vq, name, value)
    return lib


def _attention():
    q = torch.zeros(1, 2, 2, 64, dtype=torch.float16)
    vq.tree_attention(q, q, q, torch.zeros(1, 2, 32, 64, dtype=torch.float16),
                      torch.zeros(1, 2, 1, 64, 32, dtype=torch.float16), torch.zeros(1, 1, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32))


def _tree():
    vq.tree_verify(torch.zeros(1, 2, 8), None, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2),
                   torch.ones(1, 8))


@pytest.mark.parametrize("kw", ["ctx_len", "count"])
def test_append_in_place_lengths_are_refused(fake, kw):
    """Lengths updated in place would be read by some workgroups after others
    have written them."""
    k = torch.zeros(2, 2, 2, 64, dtype=torch.float16)
    lens, count = torch.zeros(2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="len_out must not be " + kw):
        vq.kv_append(k, k, torch.zeros(2, 2, 32, 64, dtype=torch.float16),
                     torch.zeros(2, 2, 1, 64, 32, dtype=torch.float16), torch.zeros(2, 1, dtype=torch.int32), lens,
                     count=count, len_out=lens if kw == "ctx_len" else count)
    assert not fake.seen


def test_verify_in_place_outputs_are_refused(fake):
    target, tokens, u, e = torch.zeros(1, 2, 8), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2), torch.ones(1, 8)
    nodes, parents = torch.ones(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    for kw in (dict(tokens_out=tokens), dict(path_out=tokens), dict(path_out=parents), dict(tokens_out=parents),
               dict(count_out=nodes)):
        with pytest.raises(ValueError, match="must not be"):
            vq.tree_verify(target, None, tokens, u, e, parents=parents, n_nodes=nodes, **kw)
    assert not fake.seen


def _greedy():
    vq.greedy_verify(torch.zeros(2, 8), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("call", [_attention, _tree, _greedy])
def test_threads_on_one_stream_do_not_interleave(fake, call):
    """These calls enqueue several kernels that pass data through the
    workspace: while one is enqueueing, no other call may be given the same
    buffer on the same stream."""
    fake.patience = 0.3
    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
        time.sleep(0.02)
    for t in threads:
        t.join()
    assert len(fake.seen) == 2 and not fake.shared


@pytest.mark.parametrize("call", [_attention, _tree, _greedy])
def test_a_replaced_buffer_is_kept(fake, call):
    """A graph captured with the cached buffer has its address in its nodes:
    when a later call needs a larger one, the memory must not be handed out
    again.  What is kept stays below what is in use."""
    call()
    first = weakref.ref(next(iter(vq._auto_ws.values())).tensor)
    sizes, held = [], []
    for need in range(1025, 40000, 1000):
        fake.need = need
        vq._ws_needs.clear()
        call()
        ws = next(iter(vq._auto_ws.values()))
        assert ws.nbytes >= need
        if ws.nbytes not in sizes:
            sizes.append(ws.nbytes)
            held.append(ws.ptr())
    gc.collect()
    assert first() is not None and len(set(held)) == len(held)
    assert len(sizes) > 2 and 1024 + sum(sizes[:-1]) <= sizes[-1]
    assert set(held) <= set(fake.seen)


def test_a_replaced_buffer_of_the_verify_gemms_is_kept(fake):
    """The same for the workspace that the verify GEMMs share per stream."""
    vq._workspace_args("auto", vq.KIND_Q4_0, 256, 256, torch.device("cpu"), STREAM)
    first = weakref.ref(next(iter(vq._auto_ws.values())).tensor)
    fake.need = 5000
    ptr, nbytes = vq._workspace_args("auto", vq.KIND_Q4_0, 512, 256, torch.device("cpu"), STREAM)
    gc.collect()
    assert nbytes >= 5000 and first() is not None and first().data_ptr() != ptr
