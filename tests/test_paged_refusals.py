"""Argument checks of the paged-cache operators, on the host: the C ABI's
documented codes (every case fails before a launch), host tensors, and the
binding's own checks of shapes, types and strides."""
import pytest
import torch

import context_exact_attention_ring_b200 as ra

E, U = ra.RING_EINVAL, ra.RING_EUNSUPPORTED
FAKE = 0x10000          # aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built():
    from context_exact_attention_ring_b200 import build
    build.build()


def call(name, base, **kw):
    assert set(kw) <= set(base), kw
    return getattr(ra.lib(), name)(*{**base, **kw}.values(), None)


EXTEND = dict(seq_lens=FAKE, new_lens=FAKE, table=FAKE, free=FAKE, n_free=FAKE, slot_map=FAKE, start=FAKE, cu=FAKE, B=2,
              W=8, ts=8, ps=16, max_free=4, max_tokens=4)
TRIM = dict(seq_lens=FAKE, keep=FAKE, table=FAKE, free=FAKE, n_free=FAKE, B=2, W=8, ts=8, ps=16, max_free=4)
APPEND = dict(k=FAKE, v=FAKE, kn=FAKE, vn=FAKE, slots=FAKE, T=3, Hkv=2, D=64, N=4, ps=16, sp=2048, st=128, sh=64, nt=128,
              nh=64, dtype=0)
DECODE = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, seq_lens=FAKE, sel=None, n_sel=None, out=FAKE, lse=FAKE, B=2, Hq=4,
              Hkv=2, D=64, N=4, ps=16, W=8, K=0, qb=256, qh=64, sp=2048, st=128, sh=64, ts=8, scale=0.1, dtype=0,
              out_dtype=0, ws=FAKE * 16, wsb=1 << 30)
BOUNDS = dict(k=FAKE, bounds=FAKE, table=FAKE, seq_lens=FAKE, start=None, B=2, Hkv=2, D=64, N=4, ps=16, W=8, sp=2048,
              st=128, sh=64, ts=8, dtype=0)
SCORES = dict(q=FAKE, bounds=FAKE, table=FAKE, seq_lens=FAKE, scores=FAKE, B=2, Hq=4, Hkv=2, D=64, N=4, ps=16, W=8,
              qb=256, qh=64, ts=8, dtype=0)
SELECT = dict(scores=FAKE, seq_lens=FAKE, sel=FAKE, n_sel=FAKE, B=2, Hkv=2, W=8, ps=16, K=4, first=1, last=1)

CASES = [("ring_attn_page_extend", EXTEND, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("seq_lens", "new_lens", "table", "free", "n_free", "slot_map", "start", "cu")],
    (dict(seq_lens=FAKE + 2), E), (dict(B=0), E), (dict(W=0), E), (dict(ts=7), E), (dict(max_free=0), E),
    (dict(max_tokens=0), E), (dict(ps=0), E), (dict(ps=-16), E), (dict(ps=12), U), (dict(ps=4), U), (dict(ps=2048), U),
    (dict(W=1 << 28, ts=1 << 28), E)]]
CASES += [("ring_attn_page_trim", TRIM, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("seq_lens", "keep", "table", "free", "n_free")],
    (dict(B=-1), E), (dict(ts=7), E), (dict(ps=24), U), (dict(max_free=0), E)]]
CASES += [("ring_attn_paged_append", APPEND, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("k", "v", "kn", "vn", "slots")],
    (dict(kn=FAKE + 8), E), (dict(T=0), E), (dict(Hkv=0), E), (dict(N=0), E), (dict(D=96), U), (dict(ps=10), U),
    (dict(dtype=5), E), (dict(st=60), E), (dict(sh=68), E), (dict(sh=32), E), (dict(nt=129), E), (dict(nh=65), E),
    (dict(N=1 << 28), E), (dict(sp=1 << 40), E)]]
CASES += [("ring_attn_decode_paged", DECODE, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("q", "k", "v", "table", "seq_lens", "out", "ws")],
    (dict(q=FAKE + 8), E), (dict(lse=FAKE + 2), E), (dict(sel=FAKE, K=2), E), (dict(n_sel=FAKE, K=2), E),
    (dict(sel=FAKE, n_sel=FAKE, K=0), E), (dict(Hq=3), E), (dict(B=0), E), (dict(D=96), U), (dict(ps=48), U),
    (dict(scale=0.0), E), (dict(scale=float("nan")), E), (dict(scale=float("inf")), E), (dict(dtype=3), E),
    (dict(out_dtype=2), E), (dict(dtype=1, out_dtype=0), U), (dict(ws=FAKE * 16 + 16), E), (dict(wsb=1000), E),
    (dict(ts=7), E), (dict(qb=257), E), (dict(qh=63), E), (dict(qh=0), E), (dict(qb=0), E), (dict(sp=0), E),
    (dict(W=1 << 27, ts=1 << 27), E), (dict(B=1 << 20, W=1 << 22, ts=1 << 22), E)]]
CASES += [("ring_attn_page_bounds", BOUNDS, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("k", "bounds", "table", "seq_lens")],
    (dict(start=FAKE + 1), E), (dict(B=0), E), (dict(B=65536), U), (dict(D=32), U), (dict(dtype=2), E), (dict(ts=1), E),
    (dict(ps=100), U)]]
CASES += [("ring_attn_page_scores", SCORES, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("q", "bounds", "table", "seq_lens", "scores")],
    (dict(Hq=5), E), (dict(D=256), U), (dict(Hq=130), U), (dict(B=40000), U), (dict(ps=7), U), (dict(qh=4), E),
    (dict(dtype=-1), E)]]
CASES += [("ring_attn_page_select", SELECT, kw, code) for kw, code in [
    *[({n: None}, E) for n in ("scores", "seq_lens", "sel", "n_sel")],
    (dict(K=0), E), (dict(first=-1), E), (dict(last=-1), E), (dict(first=3, last=2), E), (dict(W=0), E), (dict(ps=9), U)]]


@pytest.mark.parametrize("name,base,kw,code", CASES, ids=[f"{n[10:]}-{'-'.join(f'{k}={v}' for k, v in kw.items())}"
                                                         for n, _, kw, _ in CASES])
def test_abi_argument_checks(name, base, kw, code):
    assert call(name, base, **kw) == code


def test_workspace_bytes():
    assert ra.ring_attn_decode_paged_workspace_bytes(64) > 0
    assert ra.ring_attn_decode_paged_workspace_bytes(128) > ra.ring_attn_decode_paged_workspace_bytes(64)
    assert ra.ring_attn_decode_paged_workspace_bytes(96) == 0
    need = ra.ring_attn_decode_paged_workspace_bytes(64)
    assert call("ring_attn_decode_paged", DECODE, wsb=need - 1) == E


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


POOL = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
HOST = {
    "ring_attn_page_extend": lambda: ra.ring_attn_page_extend(ints(2), ints(2), ints(2, 8), ints(4), ints(1), 16, 4),
    "ring_attn_page_trim": lambda: ra.ring_attn_page_trim(ints(2), ints(2), ints(2, 8), ints(4), ints(1), 16),
    "ring_attn_paged_append": lambda: ra.ring_attn_paged_append(POOL, POOL, POOL[0], POOL[0], ints(16)),
    "ring_attn_decode_paged": lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(2, 8), ints(2)),
    "ring_attn_page_bounds": lambda: ra.ring_attn_page_bounds(POOL, ints(2, 8), ints(2)),
    "ring_attn_page_scores": lambda: ra.ring_attn_page_scores(POOL[0, :2], torch.zeros((4, 2, 2, 64), dtype=POOL.dtype),
                                                              ints(2, 8), ints(2), 16),
    "ring_attn_page_select": lambda: ra.ring_attn_page_select(torch.zeros((2, 2, 8)), ints(2), 16, 4),
}


@pytest.mark.parametrize("name", sorted(HOST))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA device"):
        HOST[name]()


@pytest.fixture
def as_if_on_gpu(monkeypatch):
    """The binding's checks with host tensors: device check and launch stubbed out."""
    calls = []
    monkeypatch.setattr(ra, "_one_device", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(ra, "_launch", lambda name, dev, *args: calls.append((name, args)))
    return calls


def test_binding_checks_shapes_types_and_strides(as_if_on_gpu):
    bad = [
        lambda: ra.ring_attn_page_extend(ints(2), ints(3), ints(2, 8), ints(4), ints(1), 16, 4),
        lambda: ra.ring_attn_page_extend(ints(2), ints(2), ints(3, 8), ints(4), ints(1), 16, 4),
        lambda: ra.ring_attn_page_extend(ints(2), ints(2), ints(2, 8), ints(4), ints(1), 16),
        lambda: ra.ring_attn_page_extend(ints(2), ints(2), ints(2, 8), ints(4), ints(1), 16, 4, slot_map=ints(5)),
        lambda: ra.ring_attn_page_extend(ints(2).long(), ints(2), ints(2, 8), ints(4), ints(1), 16, 4),
        lambda: ra.ring_attn_page_extend(ints(2), ints(2), ints(8, 2).T, ints(4), ints(1), 16, 4),
        lambda: ra.ring_attn_page_trim(ints(2), ints(2), ints(2, 8), ints(4), ints(2), 16),
        lambda: ra.ring_attn_paged_append(POOL, POOL[:3], POOL[0], POOL[0], ints(16)),
        lambda: ra.ring_attn_paged_append(POOL, POOL.float(), POOL[0], POOL[0], ints(16)),
        lambda: ra.ring_attn_paged_append(POOL, POOL, POOL[0].float(), POOL[0].float(), ints(16)),
        lambda: ra.ring_attn_paged_append(POOL, POOL, POOL[0], POOL[0], ints(15)),
        lambda: ra.ring_attn_paged_append(POOL, POOL, POOL[0], POOL[0].transpose(0, 1).contiguous().transpose(0, 1), ints(16)),
        lambda: ra.ring_attn_paged_append(POOL.transpose(2, 3), POOL.transpose(2, 3), POOL[0], POOL[0], ints(16)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(3, 8), ints(2)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2].float(), POOL, POOL, ints(2, 8), ints(2)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2, :, :32], POOL, POOL, ints(2, 8), ints(2)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(2, 8), ints(2), sel=ints(2, 2, 3)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(2, 8), ints(2), sel=ints(2, 1, 3), n_sel=ints(2, 2)),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(2, 8), ints(2), out=POOL[0, :2], out_dtype=torch.float32),
        lambda: ra.ring_attn_decode_paged(POOL[0, :2], POOL, POOL, ints(2, 8), ints(2), out_lse=torch.zeros(2, 3)),
        lambda: ra.ring_attn_page_bounds(POOL, ints(2, 8), ints(2), bounds=torch.zeros((4, 2, 2, 64))),
        lambda: ra.ring_attn_page_scores(POOL[0, :2], torch.zeros((4, 2, 2, 64)), ints(2, 8), ints(2), 16),
        lambda: ra.ring_attn_page_scores(POOL[0, :2], torch.zeros((4, 2, 3, 64), dtype=POOL.dtype), ints(2, 8), ints(2), 16),
        lambda: ra.ring_attn_page_select(torch.zeros((2, 2, 8)), ints(2), 16, 4, sel=ints(2, 2, 5)),
        lambda: ra.ring_attn_page_select(torch.zeros((2, 2, 8)).double(), ints(2), 16, 4),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
        assert not as_if_on_gpu, i


def test_binding_passes_strides_of_views(as_if_on_gpu):
    # heads before tokens, K and V side by side, a slice of a fused projection, rows of a wider table
    both = torch.zeros((4, 2, 2, 16, 64), dtype=torch.bfloat16)       # [pages, k/v, heads, tokens, D]
    k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    qkv = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    table = ints(3, 12)[:, :8]
    ra.ring_attn_decode_paged(qkv[:, :4], k, v, table, ints(3), workspace=torch.zeros(256, dtype=torch.uint8))
    name, args = as_if_on_gpu.pop()
    assert name == "ring_attn_decode_paged"
    # W, K, q strides, page / token / head strides, table stride
    assert args[15:23] == (8, 0, 512, 64, 4096, 64, 1024, 12)
    # one page, one head: their strides say nothing
    one = torch.zeros((1, 16, 1, 64), dtype=torch.float32).expand(1, 16, 1, 64)
    ra.ring_attn_paged_append(one, one, one[0], one[0], ints(16))
    name, args = as_if_on_gpu.pop()
    assert args[10:15] == (1024, 64, 64, 64, 64)


PACKED = [("ring_attn_page_extend", EXTEND), ("ring_attn_page_trim", TRIM), ("ring_attn_paged_append", APPEND),
          ("ring_attn_decode_paged", DECODE), ("ring_attn_page_bounds", BOUNDS), ("ring_attn_page_scores", SCORES),
          ("ring_attn_page_select", SELECT)]


@pytest.mark.parametrize("i,name,base", [(i, n, b) for i, (n, b) in enumerate(PACKED)])
def test_packed_calls_take_their_arguments_in_order(i, name, base):
    # every argument that the flat call refuses is refused in its place of the packed words
    import ctypes
    call_no, words, n = ra._PACKED[name]
    assert call_no == i and n == len(base) == words.size // 8
    assert len(ra._PACKED) == len(PACKED)
    fn = ra.lib().ring_attn_paged_packed
    for nm, b, kw, code in CASES:
        if nm == name:
            packed = words.pack(*[0 if v is None else v for v in {**b, **kw}.values()])
            assert fn(i, packed, n, None) == code, kw
    packed = words.pack(*[0 if v is None else v for v in base.values()])
    assert fn(i, packed, n - 1, None) == E and fn(i, None, n, None) == E
    assert fn(len(PACKED), packed, n, None) == E and fn(-1, packed, n, None) == E
    buf = ctypes.create_string_buffer(packed + b"\0" * 16)
    at = ctypes.addressof(buf)
    assert fn(i, at + 4 - at % 4, n, None) == E if (at + 4 - at % 4) % 8 else True


class _Fake:
    def __init__(self, dev):
        self.dev = dev

    def get_device(self):
        return self.dev


def test_tensors_of_one_device_and_its_stream(monkeypatch):
    assert ra._one_device(_Fake(1), None, _Fake(1)) == 1
    for devs in ((0, 1), (-1,), (0, -1), (-1, 0)):
        with pytest.raises(ValueError, match="device"):
            ra._one_device(*(_Fake(d) for d in devs))
    # a call on tensors of another device than the current one switches to it, and takes its stream
    import contextlib
    seen, current = [], [0]

    class Lib:
        def ring_attn_paged_packed(self, call, words, n, stream):
            seen.append((call, n, stream, current[0]))
            return 0

    @contextlib.contextmanager
    def device(d):
        old, current[0] = current[0], d
        yield
        current[0] = old

    monkeypatch.setattr(ra, "_lib", Lib())
    monkeypatch.setattr(ra, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    ra._launch("ring_attn_page_select", 0, *range(11))
    ra._launch("ring_attn_page_select", 2, *range(11))
    assert seen == [(6, 11, 1000, 0), (6, 11, 1002, 2)] and current == [0]
