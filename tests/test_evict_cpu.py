"""The host side of eviction without a device: what is refused before a GPU is touched, and which tensors a call
holds back for the stream it runs on (the C entry points and torch's streams are replaced by fakes)."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import SharedKVPool, eviction
from cross_model_shared_gb300 import _native as N
from cross_model_shared_gb300 import build as B

OWN = ("k_pages", "v_pages", "block_table", "seq_lens", "error_word")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load()


def test_null_pools(lib):
    bad = N.SHKV_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    m = N.shkv_mass(16, 1, 1, 1)
    r = ctypes.byref(m)
    assert lib.shkv_decode_mass(None, 1, 1, 1, 16, 1.0, 16, 1.0, r, r, None) == bad
    assert lib.shkv_prefill_mass(None, 1, 1, 1, 16, 64, 64, 1.0, 16, 1, 1, 1.0, r, r, 16, 1 << 20, None) == bad
    assert lib.shkv_prefill_mass_workspace_size(None, ctypes.byref(n)) == bad
    assert lib.shkv_select_width(None, 1, None, ctypes.byref(ctypes.c_int32())) == bad
    assert lib.shkv_select_tokens(None, 1, r, None, 0, 0, 16, 1, None) == bad
    assert lib.shkv_evict_tokens(None, 1, None, 16, 1, 16, 1, None, 0, None, None, None, None) == bad


class Fake:
    """Records what was held back for which stream, and when the entry points were called."""

    def __init__(self):
        self.events, self.raw, self.capturing = [], 7, False

    def entry(self, name):
        return lambda *a: self.events.append(name)

    def held(self):
        return [e[1:] for e in self.events if e[0] == "hold"]


class Watched(torch.Tensor):
    def record_stream(self, stream):
        self.fake.events.append(("hold", self.label, stream))


def watched(fake, name, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Watched)
    t.fake, t.label = fake, name
    return t


@pytest.fixture
def fake(monkeypatch):
    f = Fake()
    for name in ("decode_mass", "prefill_mass", "select_tokens", "evict_tokens"):
        monkeypatch.setattr(eviction.N, f"shkv_{name}", f.entry(name))
    monkeypatch.setattr(eviction.N, "shkv_prefill_mass_workspace_size", lambda pool: 64)

    monkeypatch.setattr(eviction.N, "shkv_select_width", lambda pool, n, keep: 9)
    monkeypatch.setattr(eviction, "_raw_stream", lambda index: f.raw)
    monkeypatch.setattr(eviction, "_current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: f"stream {f.raw}")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: f.capturing)
    return f


@pytest.fixture
def pool(fake):
    p = object.__new__(SharedKVPool)
    p.num_kv_heads, p.head_dim, p.page_size, p.max_batch, p.max_pages_per_seq, p.handle = 2, 64, 16, 4, 4, None
    for name in OWN:
        setattr(p, name, watched(fake, name, 4))
    return p


def calls(fake, pool):
    f32, i32 = torch.float32, torch.int32
    q, lse = watched(fake, "q", 3, 8, 64), watched(fake, "lse", 3, 8, dtype=f32)
    qp, lp = watched(fake, "q", 3, 5, 4, 64), watched(fake, "lse", 3, 5, 4, dtype=f32)
    mass, out = (watched(fake, n, 3, 2, 20, dtype=f32) for n in ("mass", "out"))
    index, new, table = (watched(fake, n, *s, dtype=i32) for n, s in (("index", (3, 2, 9)), ("new", (3, 1)), ("table", (3, 2))))
    picked = watched(fake, "out", 3, 2, 9, dtype=i32)
    return {
        "decode_mass": (lambda: pool.decode_mass(q, lse, 2, mass, out=out), ["q", "lse", "mass", "out"]),
        "prefill_mass": (lambda: pool.prefill_mass(qp, lp, mass, out=out), ["q", "lse", "mass", "out"]),
        "select_tokens": (lambda: pool.select_tokens(mass, [9, 9, 9], out=picked), ["mass", "out"]),
        "evict_tokens": (lambda: pool.evict_tokens(index, [9, 9, 9], new, mass=mass, out=out, source=(table, [20] * 3)),
                         ["index", "new", "table", "mass", "out"]),
    }


NAMES = ["decode_mass", "prefill_mass", "select_tokens", "evict_tokens"]


@pytest.mark.parametrize("name", NAMES)
def test_a_calls_tensors_are_held_for_the_side_stream_that_is_current(fake, pool, name):
    call, tensors = calls(fake, pool)[name]
    for _ in range(2):
        del fake.events[:]
        call()
        assert fake.events[-1] == name                           # ... before its kernels are enqueued
        assert set(fake.held()) >= {(t, "stream 7") for t in tensors}


def test_and_for_the_default_stream_where_it_is_named(fake, pool, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    fake.raw = 0
    named = type("Stream", (), {"device": pool.k_pages.device, "cuda_stream": 0})()
    mass = watched(fake, "mass", 3, 2, 20, dtype=torch.float32)
    pool.select_tokens(mass, [9, 9, 9], stream=named)
    assert {t for t, _ in fake.held()} == {"mass", *OWN}
    other = type("Stream", (), {"device": torch.device("meta"), "cuda_stream": 0})()
    with pytest.raises(ValueError):
        pool.select_tokens(mass, [9, 9, 9], stream=other)


def test_on_the_default_stream_tensors_are_the_callers(fake, pool):
    fake.raw = 0
    for call, _ in calls(fake, pool).values():
        call()
    assert {t for t, _ in fake.held()} == set(OWN)


def test_the_pools_memory_is_held_once_for_every_stream(fake, pool):
    for raw in (0, 7, 0, 9, 7):
        fake.raw = raw
        for call, _ in calls(fake, pool).values():
            call()
    for name in OWN:
        assert sorted(s for t, s in fake.held() if t == name) == ["stream 0", "stream 7", "stream 9"]


def test_nothing_is_held_while_a_graph_is_captured_and_scratch_is_its_own(fake, pool):
    fake.capturing = True
    for call, _ in calls(fake, pool).values():
        call()
    assert not fake.held() and not pool._mass_workspaces
    fake.capturing = False
    calls(fake, pool)["prefill_mass"][0]()
    kept = pool._mass_workspaces[7]
    fake.capturing = True
    calls(fake, pool)["prefill_mass"][0]()
    assert pool._mass_workspaces == {7: kept}


def bad_calls(fake, pool):
    f32, i32, bf = torch.float32, torch.int32, torch.bfloat16
    z = torch.zeros
    q, lse, mass = z(3, 8, 64, dtype=bf), z(3, 8), z(3, 2, 20)
    qp, lp = z(3, 5, 4, 64, dtype=bf), z(3, 5, 4)
    index, new = z(3, 2, 9, dtype=i32), z(3, 1, dtype=i32)
    d, p, s, e = pool.decode_mass, pool.prefill_mass, pool.select_tokens, pool.evict_tokens
    k = [9, 9, 9]
    return [
        lambda: d(q.half(), lse, 2, mass), lambda: d(q[0], lse, 2, mass), lambda: d(q[:, ::2], lse[:, ::2], 2, mass),
        lambda: d(q, lse, 3, mass), lambda: d(q, lse, 0, mass), lambda: d(z(3, 8, 128, dtype=bf), lse, 2, mass),
        lambda: d(q, lse.double(), 2, mass), lambda: d(q, lse[:, :4], 2, mass), lambda: d(q, lse, 2, mass.double()),
        lambda: d(q, lse, 2, mass[0]), lambda: d(q, lse, 2, mass[:2]), lambda: d(q, lse, 2, mass[:, :1]),
        lambda: d(q, lse, 2, z(3, 2, 40)[:, :, ::2]), lambda: d(q, lse, 2, mass, out=z(3, 2, 20, dtype=i32)),
        lambda: d(z(5, 8, 64, dtype=bf), z(5, 8), 2, None), lambda: d(q.to("meta"), lse, 2, mass),
        lambda: p(qp.half(), lp, mass), lambda: p(qp[0], lp[0], mass), lambda: p(qp[..., :32], lp, mass),
        lambda: p(qp.transpose(2, 3).contiguous().transpose(2, 3), lp, mass),
        lambda: p(z(3, 5, 8, 64, dtype=bf)[:, :, ::2], lp, mass), lambda: p(qp, lp[:, :4], mass),
        lambda: p(qp, z(3, 5, 8)[:, :, ::2], mass), lambda: p(qp, lp.double(), mass),
        lambda: s(mass, [9, -1, 9]), lambda: s(mass, [9] * 4), lambda: s(mass.double(), k), lambda: s(mass, k, sink=-1),
        lambda: s(mass, k, recent=2 ** 31), lambda: s(mass, k, sink=2 ** 32 + 1), lambda: s(mass, 9),
        lambda: s(mass, k, out=index.long()), lambda: s(mass, k, out=index[:2]), lambda: s(mass, k, out=index[:, :, ::2]),
        lambda: s(z(5, 2, 20), [9] * 5),
        lambda: e(index.long(), k, new), lambda: e(index[:2], k, new), lambda: e(index[:, :1], k, new),
        lambda: e(index[0], k, new), lambda: e(index[:, :, ::2], k, new), lambda: e(index, k, new.long()),
        lambda: e(index, k, new[:2]), lambda: e(index, k, new[0]), lambda: e(index, k, new, out=mass),
        lambda: e(index, k, new, mass=mass[:2]), lambda: e(index, k, new, source=(new, [20, 20])),
        lambda: e(index, k, new, source=(new.long(), [20] * 3)), lambda: e(index, [9, 9, 2 ** 31], new),
        lambda: e(index, np.zeros((3, 1), np.int32), new),
    ]


def test_refusals_before_any_call(fake, pool):
    for i, f in enumerate(bad_calls(fake, pool)):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    assert not [e for e in fake.events if e in NAMES]
