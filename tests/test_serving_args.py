"""What the serving entry points refuse on the host, before anything touches the GPU (no GPU needed)."""
import ctypes

import pytest

INVALID, WORKSPACE = 1, 3
I32, I64, F32, PTR, SIZE = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
P = 1 << 20  # a pointer that is never followed: aligned, not null


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_seq_gb300 import build
    return ctypes.CDLL(build.build())


def call(lib, name, types, args, **changed):
    f = getattr(lib, name)
    f.restype, f.argtypes = I32, [t for _, t in types]
    return f(*[changed.get(k, args[k]) for k, _ in types])


PLAN = [("R", I32), ("page", I32), ("max_pages", I32), ("n_free", I32), ("capacity", I32)] + \
    [(n, PTR) for n in ("cached", "new", "free", "table", "q_start", "kv_len", "positions", "slots", "used", "ws")] + \
    [("bytes", SIZE), ("stream", PTR)]
PLAN_ARGS = {n: P if t is PTR else 16 for n, t in PLAN} | {"bytes": 256, "stream": None}


@pytest.mark.parametrize("changed", [dict(R=0), dict(R=-1), dict(page=0), dict(max_pages=0), dict(n_free=-1), dict(capacity=-1)] +
                         [{n: None} for n in ("cached", "new", "free", "table", "q_start", "kv_len", "positions", "slots", "used")])
def test_page_plan_refuses(lib, changed):
    assert call(lib, "dspark_page_plan", PLAN, PLAN_ARGS, **changed) == INVALID


APPEND = [("T", I32), ("Hkv", I32), ("D", I32), ("dtype", I32), ("k", PTR), ("v", PTR), ("slots", PTR), ("n_slots", I64),
          ("k_cache", PTR), ("v_cache", PTR), ("ws", PTR), ("bytes", SIZE), ("stream", PTR)]
APPEND_ARGS = {n: P if t is PTR else 8 for n, t in APPEND} | {"dtype": 1, "bytes": 256, "stream": None}


@pytest.mark.parametrize("changed", [dict(T=-1), dict(Hkv=0), dict(D=0), dict(dtype=7), dict(n_slots=-1), dict(Hkv=1 << 13, D=1 << 13)] +
                         [{n: None} for n in ("k", "v", "slots", "k_cache", "v_cache")])
def test_kv_append_refuses(lib, changed):
    assert call(lib, "dspark_kv_append", APPEND, APPEND_ARGS, **changed) == INVALID


ATTN = [(n, I32) for n in ("R", "T", "Hq", "Hkv", "D", "page", "n_pages", "max_pages", "prefix_len")] + \
    [(n, PTR) for n in ("q", "k", "v", "prefix_pages", "table", "q_start", "kv_len")] + \
    [("scale", F32), ("out", PTR), ("lse", PTR), ("ws", PTR), ("bytes", SIZE), ("stream", PTR)]
ATTN_ARGS = {n: P if t is PTR else 8 for n, t in ATTN} | {"Hkv": 2, "D": 64, "page": 16, "scale": 0.125, "bytes": 1 << 40,
                                                        "stream": None}


@pytest.mark.parametrize("changed", [
    dict(R=0), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hq=258), dict(D=96), dict(D=32), dict(page=8),
    dict(page=24), dict(page=8192), dict(n_pages=0), dict(max_pages=0), dict(prefix_len=-1), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 28), dict(q=P + 8), dict(k=P + 2), dict(v=P + 4),
    dict(out=P + 8)] + [{n: None} for n in ("q", "k", "v", "prefix_pages", "table", "q_start", "kv_len", "out")])
def test_attention_refuses(lib, changed):
    assert call(lib, "dspark_prefix_attention", ATTN, ATTN_ARGS, **changed) == INVALID


def test_attention_workspace_size(lib):
    f = lib.dspark_attention_workspace_bytes
    f.restype = SIZE
    base = f(8, 8, 8, 2, 64)
    assert base > 0 and base % 256 == 0 and f(8, 9, 8, 2, 64) > base and f(9, 8, 8, 2, 64) >= base
    for bad in ((0, 8, 8, 2, 64), (8, -1, 8, 2, 64), (8, 8, 7, 2, 64), (8, 8, 8, 0, 64), (8, 8, 8, 2, 80)):
        assert f(*bad) == 0
    assert call(lib, "dspark_prefix_attention", ATTN, ATTN_ARGS, bytes=base - 1) == WORKSPACE


RULE = [("N", I32), ("V", I32), ("dtype", I32)] + [(n, PTR) for n in ("logits", "temperature", "top_k", "top_p", "min_p")]
TAIL = [("ws", PTR), ("bytes", SIZE), ("stream", PTR)]
SAMPLE = RULE + [("u", PTR), ("tokens", PTR), ("prob", PTR)] + TAIL
TRUNCATE = RULE + [("out", PTR)] + TAIL


@pytest.mark.parametrize("name,types,own", [("dspark_sample", SAMPLE, ("u", "tokens")), ("dspark_truncate", TRUNCATE, ("out",))])
def test_rule_refuses(lib, name, types, own):
    args = {n: P if t is PTR else 8 for n, t in types} | {"dtype": 1, "bytes": 256, "stream": None}
    for changed in [dict(N=-1), dict(V=0), dict(V=(1 << 20) + 1), dict(dtype=7)] + \
            [{n: None} for n in ("logits", "temperature", "top_k", "top_p", "min_p") + own]:
        assert call(lib, name, types, args, **changed) == INVALID, changed
    # nothing to do is no error, whatever the pointers
    nothing = {n: None if t is PTR and n != "ws" else args[n] for n, t in types}
    assert call(lib, name, types, nothing, N=0) == 0


@pytest.mark.parametrize("name,types,args", [
    ("dspark_page_plan", PLAN, PLAN_ARGS), ("dspark_kv_append", APPEND, APPEND_ARGS), ("dspark_prefix_attention", ATTN, ATTN_ARGS),
    ("dspark_sample", SAMPLE, {n: P if t is PTR else 8 for n, t in SAMPLE} | {"dtype": 1, "stream": None}),
    ("dspark_truncate", TRUNCATE, {n: P if t is PTR else 8 for n, t in TRUNCATE} | {"dtype": 1, "stream": None})])
@pytest.mark.parametrize("changed", [dict(ws=None), dict(ws=P + 128), dict(bytes=255)])
def test_workspace_refused(lib, name, types, args, changed):
    assert call(lib, name, types, args, **changed) == WORKSPACE
