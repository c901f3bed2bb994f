"""Calls on a given stream take their memory from that stream (CPU only: the
library and the allocator are fakes that record what is asked of them)."""

import contextlib
import types

import pytest
import torch

import block_decoding_gb300 as bd

B = bd._binding


class Stream:
    cuda_stream = 77
    device = torch.device("cpu")


class World:
    """Which stream was current at every allocation, and what was launched where."""

    def __init__(self, mp):
        self.caller, self.side = Stream(), Stream()
        self.now = self.caller
        self.blocks, self.recorded, self.launched = {}, [], []
        empty = torch.empty

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s
            yield
            self.now = before

        def record(t, s):
            self.recorded.append((t.data_ptr(), s))

        def new(*a, **kw):
            t = empty(*a, **kw)
            self.blocks[t.data_ptr()] = self.now
            self.keep.append(t)
            return t

        self.keep = []
        mp.setattr(torch, "empty", new)
        mp.setattr(torch.cuda, "stream", stream)
        mp.setattr(torch.cuda, "current_stream", lambda *a: self.now)
        mp.setattr(torch.Tensor, "record_stream", record)
        mp.setattr(B, "_ptr", lambda t, *a: None if t is None else t.data_ptr())
        mp.setattr(B, "_ptr_on", lambda t, *a: t.data_ptr())
        mp.setattr(B, "_rows_ptr", lambda t, *a: (t.data_ptr(), t.stride(0)))
        mp.setattr(B, "_launch", lambda what, index, stream, *a: self.launched.append((what, stream)))
        mp.setattr(B, "_stream", lambda s: self.launched.append(s))
        # workspaces of 4096 bytes, every call succeeds
        mp.setattr(B, "LIB", types.SimpleNamespace(**{
            name: lambda *a, n=4096 if name.endswith("_workspace") else 0: n for name in B.SIGNATURES}))

    def check(self, returned, stream, scratch):
        """Everything allocated belongs to `stream`; what is returned, and nothing else, is kept for the caller's."""
        assert self.blocks and set(self.blocks.values()) == {stream or self.caller}
        out = {t.data_ptr() for t in returned}
        assert len(self.blocks) == len(out) + scratch
        kept = {p for p, s in self.recorded if s is self.caller}
        assert len(self.recorded) == len(kept) == (len(out) if stream else 0)
        assert not stream or kept == out


@pytest.fixture
def world(monkeypatch):
    w = types.SimpleNamespace()
    zeros = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    w.i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    w.zeros = zeros
    w.pages = types.SimpleNamespace(index=0, device=torch.device("cpu"), heads=2, dh=64, desc=B.KvPagesDesc(), _need={})
    w.w = World(monkeypatch)
    return w


@pytest.mark.parametrize("side", [False, True])
def test_paged_calls_allocate_on_their_stream(world, side):
    w = world.w
    stream = w.side if side else None
    table = torch.zeros((1, 2), dtype=torch.int32)
    out = bd.paged_attn(world.zeros(3, 4, 64), world.pages, world.i32(0, 3), world.i32(20), table, 3, 20, return_lse=True,
                        stream=stream)
    w.check(out, stream, 1)
    w.blocks.clear(), w.recorded.clear()
    w.check(bd.kv_read(world.pages, world.i32(0, 3), world.i32(0), table, 3, stream=stream), stream, 0)
    assert w.launched == [("dllm_paged_attn", stream), ("dllm_kv_read", stream)]


@pytest.mark.parametrize("side", [False, True])
def test_other_calls_allocate_on_their_stream(world, side):
    w, z, i32 = world.w, world.zeros, world.i32
    stream = w.side if side else None
    params = dict(tau=0.9, lam=0.5, kappa=0.1, hierarchical=1, hier_levels=2, smoothing=1, alpha=0.5, mask_id=0)
    f32 = lambda *s: z(*s, t=torch.float32)  # noqa: E731
    byte = lambda *s: z(*s, t=torch.uint8)  # noqa: E731
    desc, keep = B.ModelDesc(), [z(4, 64)]
    calls = [
        (lambda: [bd.block_attn(z(3, 2, 64), z(5, 2, 64), z(5, 2, 64), i32(0, 3), i32(0, 5), 3, 5, stream=stream)], 1),
        (lambda: bd.head_confidence(z(3, 64), z(32, 64), z(32, 64), stream=stream), 1),
        (lambda: bd.commit(i32(0, 1), f32(2), None, i32(0, 0), i32(0, 1), byte(1, 2), i32(0, 0), f32(2), i32(0, 0),
                           z(32, 64), params, stream=stream), 0),
        (lambda: [bd.gemm_bf16(z(3, 64), z(8, 64), stream=stream)], 0),
        (lambda: [bd.model_forward(desc, z(4, 64), 0, keep, keep, stream=stream)], 1),
        (lambda: bd.moe_ffn(z(3, 64), z(4, 64), z(4, 32, 64), z(4, 64, 16), 2, stream=stream), 1),
    ]
    for call, scratch in calls:
        w.blocks.clear(), w.recorded.clear()
        w.check(call(), stream, scratch)
    assert w.launched == [stream] * len(calls)


@pytest.mark.parametrize("side", [False, True])
def test_a_served_step_stays_on_its_stream(monkeypatch, side):
    """The plan's upload, the step and the read of its commit counts."""
    from block_decoding_gb300 import serve

    class Ordered(Stream):
        def __init__(self, log):
            self.log = log

        def wait_stream(self, other):
            self.log.append(("wait", self, other))

        def synchronize(self):
            self.log.append(("sync", self))

    log = []
    caller, given = Ordered(log), Ordered(log)
    now = [caller]

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    copy = torch.Tensor.copy_
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
    monkeypatch.setattr(torch.Tensor, "copy_", lambda t, *a, **kw: (log.append(("copy", now[-1])), copy(t, *a, **kw))[1])
    monkeypatch.setattr(serve.B, "step_args", lambda **kw: None)
    monkeypatch.setattr(serve.B, "denoise_step_workspace", lambda a: 256)
    monkeypatch.setattr(serve.B, "denoise_step", lambda a, ws, s=None: log.append(("step", s or now[-1])))
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    bufs = dict(q=z(200, 1, 64), k=z(200, 1, 64), v=z(200, 1, 64), w_head=z(32, 64), emb=z(32, 64), hidden=z(16, 64))
    srv = serve.StepServer(bufs, slots=2, blk=8, vic=0, params=dict(mask_id=0, smoothing=0), quantum=100, budget_cap=200,
                           max_step_rows=100, max_seq=64, device="cpu")
    assert srv.submit(0, 16, 8)
    del log[:]
    assert srv.step(given if side else None)
    on = given if side else caller
    assert [x for x in log if x[0] != "wait"] == [("copy", on), ("step", on), ("copy", on), ("sync", on)]
    assert [x for x in log if x[0] == "wait"] == ([("wait", given, caller)] if side else [])
