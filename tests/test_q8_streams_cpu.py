"""Which tensors the 8-bit cache's Python calls hold back for the stream they run on, without a device: the C
entry points and torch's streams are replaced by fakes."""
import pytest
import torch

from cross_model_shared_gb300 import q8


OWN = ("k_pages", "v_pages", "scales", "block_table", "seq_lens", "error_word")


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


@pytest.fixture
def fake(monkeypatch):
    f = Fake()
    for name in ("append_kv", "read_kv", "decode_attention", "chunk_attention"):
        monkeypatch.setattr(q8.N, f"shkv_q8_{name}", f.entry(name))
    monkeypatch.setattr(q8, "_raw_stream", lambda index: f.raw)
    monkeypatch.setattr(q8, "_current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: f"stream {f.raw}")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: f.capturing)
    return f


@pytest.fixture
def pool(fake):
    p = object.__new__(q8.QuantizedKVPool)
    p.device = torch.device("cpu")
    p.num_kv_heads, p.head_dim, p.page_size, p.max_batch, p.max_pages_per_seq = 2, 64, 16, 4, 4
    p.handle, p.workspace_bytes, p.workspace_zero_bytes = None, 64, 16
    p._workspaces, p._streams = {}, {}
    for name in OWN:
        setattr(p, name, watched(fake, name, 4))
    return p


def watched(fake, name, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Watched)
    t.fake, t.label = fake, name
    return t


def calls(fake, pool):
    kv = lambda name: watched(fake, name, 3, 2, 64)             # noqa: E731
    q = lambda name: watched(fake, name, 3, 4, 64)              # noqa: E731
    lse = watched(fake, "lse", 3, 4, dtype=torch.float32)
    ws = watched(fake, "workspace", 64, dtype=torch.uint8)
    return {
        "append_kv": (lambda: pool.append_kv(kv("k"), kv("v"), [3]), ["k", "v"]),
        "read_kv": (lambda: pool.read_kv([0], [3], k_out=kv("k"), v_out=kv("v")), ["k", "v"]),
        "decode_attention": (lambda: pool.decode_attention(q("q"), 2, out=q("out"), lse=lse, workspace=ws),
                             ["q", "out", "lse", "workspace"]),
        "chunk_attention": (lambda: pool.chunk_attention(q("q"), [3], out=q("out"), lse=lse, workspace=ws),
                            ["q", "out", "lse", "workspace"]),
    }


@pytest.mark.parametrize("name", ["append_kv", "read_kv", "decode_attention", "chunk_attention"])
def test_a_calls_tensors_are_held_for_the_side_stream_that_is_current(fake, pool, name):
    call, tensors = calls(fake, pool)[name]
    for _ in range(2):
        del fake.events[:]
        call()
        assert fake.events[-1] == name                          # ... before its kernels are enqueued
        assert set(fake.held()) >= {(t, "stream 7") for t in tensors}


def test_and_for_the_default_stream_where_it_is_named(fake, pool, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: q8._HERE)
    fake.raw = 0
    named = type("Stream", (), {"device": pool.device, "cuda_stream": 0})()
    pool.append_kv(watched(fake, "k", 3, 2, 64), watched(fake, "v", 3, 2, 64), [3], stream=named)
    assert {t for t, _ in fake.held()} == {"k", "v", *OWN}


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
    first = fake.events.index("append_kv")
    assert {t for t, _ in [e[1:] for e in fake.events[:first]]} >= set(OWN)


def test_nothing_is_held_while_a_graph_is_captured(fake, pool):
    fake.capturing = True
    for call, _ in calls(fake, pool).values():
        call()
    assert not fake.held()
