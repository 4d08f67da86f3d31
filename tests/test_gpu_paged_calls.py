"""GPU tests of the paged calls' native argument checks: they answer None (and launch nothing) to what
the binding's own checks refuse, which then say why; both ways make the same call."""
import pytest
import torch

import prefill_only_cascade_gb300 as q

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(q._calls is None, reason="built without PyTorch's or Python's headers")]
DEV, BF, I32, F32, U8 = "cuda", torch.bfloat16, torch.int32, torch.float32, torch.uint8
NATIVE = {"append": q.paged_kv_append, "read": q.paged_kv_read, "decode": q.paged_decode_attn,
          "evict": q.paged_kv_evict}


@pytest.fixture(autouse=True)
def no_device_error():
    q.get_device_error()
    yield
    assert q.get_device_error() == q.QUAIL_OK


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def arguments(form):
    """Arguments of the four calls by name, in the order of the functions' own."""
    B, hkv, hq, d, page = 2, 2, 8, 64, 16
    desc = q.make_paged_desc(B, 40, 6, page, 3, hq, hkv, d, kv_fp8=form == "fp8", kv_fp4=form == "fp4")
    dtype = {"bf16": BF, "fp8": torch.float8_e4m3fn, "fp4": U8}[form]
    pool = lambda n: torch.zeros(q.paged_pool_shape(desc, n), dtype=dtype, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=I32, device=DEV)
    k, v, table = pool(6), pool(6), i32(5, 0, 3, 1, 2, 4).view(2, 3)
    scale = dict(k_scale=torch.full((B, hkv), 0.01, device=DEV), v_scale=torch.full((B, hkv), 0.02, device=DEV))
    if form == "bf16":
        scale = dict(k_scale=None, v_scale=None)
    rows = [randn(60, hkv, d, seed=i) for i in range(2)]
    ws = lambda n: torch.empty(max(n, 16), dtype=U8, device=DEV)
    return {
        "append": dict(desc=desc, k_new=rows[0], v_new=rows[1], start_pos=i32(0, 0), block_table=table,
                       k_pages=k, v_pages=v, new_offsets=i32(0, 40, 60), **scale),
        "read": dict(desc=desc, k_pages=k, v_pages=v, start_pos=i32(0, 0), block_table=table,
                     k_out=torch.empty_like(rows[0]), v_out=torch.empty_like(rows[0]), offsets=i32(0, 40, 60),
                     **scale),
        "decode": dict(desc=desc, q=randn(B, hq, d, seed=3), k_pages=k, v_pages=v, block_table=table,
                       seq_lens=i32(40, 20), out=torch.empty(B, hq, d, dtype=BF, device=DEV),
                       workspace=ws(q.paged_decode_workspace_size(desc, True)),
                       lse=torch.empty(B, hq, device=DEV), **scale, score_in=torch.ones(B, hkv, 41, device=DEV),
                       score_out=torch.zeros(B, hkv, 41, device=DEV)),
        "evict": dict(desc=desc, budget=20, recent=4, k_pages=k, v_pages=v, block_table=table,
                      seq_lens=i32(40, 20), score=torch.rand(B, hkv, 40, device=DEV), dst_table=i32(0, 1, 2, 3).view(2, 2),
                      k_dst=pool(4), v_dst=pool(4), kept=torch.zeros(B, hkv, 20, dtype=I32, device=DEV),
                      new_lens=i32(0, 0), workspace=ws(q.paged_evict_workspace_size(desc, 4)),
                      score_out=torch.zeros(B, hkv, 20, device=DEV)),
    }


OUTPUTS = {"append": ("k_pages", "v_pages"), "read": ("k_out", "v_out"), "decode": ("out", "lse", "score_out"),
           "evict": ("k_dst", "v_dst", "kept", "new_lens", "score_out")}


def native(name, args):
    return getattr(q._calls, name)(*args.values())


@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
def test_both_ways_make_the_same_call(form):
    got = {}
    for stream in (None, torch.cuda.current_stream()):   # native, and the binding's own checks
        calls = arguments(form)
        for name, call in NATIVE.items():
            if stream is None:
                assert native(name, calls[name]) == q.QUAIL_OK
            else:
                call(**calls[name], stream=stream)
            if name == "append":                         # the others take what it wrote
                for other in ("read", "decode", "evict"):
                    calls[other]["k_pages"], calls[other]["v_pages"] = calls[name]["k_pages"], calls[name]["v_pages"]
            got.setdefault(name, []).append([calls[name][o].float() for o in OUTPUTS[name]])
    for name, (a, b) in got.items():
        if name != "evict":
            assert all(torch.equal(x, y) for x, y in zip(a, b)), name


def wrong(t):
    """Tensors like t that the calls refuse."""
    yield t.cpu()
    yield t.double() if t.dtype is not U8 else t.to(torch.int8)
    yield t[:-1]
    yield t[None]
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=DEV)
    yield wide[..., ::2]


@pytest.mark.parametrize("form", ["bf16", "fp4"])
@pytest.mark.parametrize("name", NATIVE)
def test_refusals(name, form):
    args = arguments(form)[name]
    for key, value in args.items():
        bad = [3, "x"]
        if isinstance(value, torch.Tensor):
            bad += [w for w in wrong(value) if not (key in ("workspace", "k_dst", "v_dst") and w.shape != value.shape)]
            if key not in ("new_offsets", "offsets", "lse", "score_in", "score_out", "k_out", "v_out"):
                bad.append(None)
        elif key in ("budget", "recent"):
            bad = [2 ** 31, -2 ** 40, None, "x"]
        elif value is None:
            bad = [torch.ones(2, 2, device=DEV)]
        for x in bad:
            these = {**args, key: x}
            if key == "workspace" and isinstance(x, torch.Tensor) and x.dtype is U8 and x.is_cuda and x.dim() == 1 \
                    and x.is_contiguous():
                continue
            before = [args[o].clone() for o in OUTPUTS[name]]
            assert native(name, these) is None, (key, x)
            with pytest.raises((TypeError, ValueError, AttributeError, q.QuailError)):
                NATIVE[name](**these)
            assert all(torch.equal(a.view(U8) if a.dtype is BF else a, b.view(U8) if b.dtype is BF else b)
                       for a, b in zip(before, (args[o] for o in OUTPUTS[name])))


def test_numbers_of_arguments_and_status():
    args = arguments("fp4")
    assert q._calls.append() is None and q._calls.decode(*list(args["decode"].values())[:5]) is None
    short = {**args["decode"], "workspace": torch.empty(16, dtype=U8, device=DEV)}
    assert native("decode", short) == q.QUAIL_ERR_INVALID_ARG
    with pytest.raises(q.QuailError):
        q.paged_decode_attn(**short)
    with pytest.raises(TypeError):
        q._calls.bind(1, 2)
