"""The paged 8-bit cache operators refuse bad arguments on the host, before any CUDA call (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import dsa_lightning_indexer_02_b200 as dsa

lib = dsa.lib()
P = ctypes.c_void_p
A, A2, M, ODD = P(0x10000), P(1 << 40), P(0x10004), P(0x10002)
INV, UNS, WS = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE
NAN = float("nan")


def rope(x=A, dtype=0, T=4, H=2, D=128, x_ts=256, x_hs=128, pos=None, pos0=0, inv=A, off=0, R=64, layout=0, m=1.0,
         inverse=0, out=A2, o_ts=256, o_hs=128):
    return lib.dsa_rope(x, dtype, T, H, D, x_ts, x_hs, pos, pos0, inv, off, R, layout, m, inverse, out, o_ts, o_hs, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), INV), (dict(out=None), INV), (dict(inv=None), INV), (dict(x=M), INV), (dict(out=M), INV),
    (dict(inv=M), INV), (dict(pos=ODD), INV), (dict(dtype=2), INV), (dict(layout=2), INV), (dict(T=0), INV),
    (dict(H=0), INV), (dict(R=0), INV), (dict(R=-16), INV), (dict(off=-8), INV), (dict(off=72), INV), (dict(m=NAN), INV),
    (dict(x_ts=-256), INV), (dict(x_ts=260), INV), (dict(o_hs=132), INV), (dict(o_ts=248), INV), (dict(o_ts=0), INV),
    (dict(o_hs=64), INV), (dict(pos0=1 << 31), INV), (dict(pos0=(1 << 31) - 3), INV), (dict(x_ts=1 << 41), INV),
    (dict(out=A, o_ts=512), INV),                       # the same memory, other strides
    (dict(out=P(0x10000 + 256)), INV), (dict(x=P((1 << 40) + 2032)), INV),   # overlapping ranges
    (dict(D=132, x_hs=136, o_hs=136, x_ts=272, o_ts=272), UNS), (dict(R=24), UNS), (dict(off=4), UNS),
    (dict(D=520, x_hs=520, o_hs=520, x_ts=1040, o_ts=1040), UNS), (dict(H=5000, x_ts=640000, o_ts=640000), UNS),
    (dict(D=512, R=272, x_hs=512, o_hs=512, x_ts=1024, o_ts=1024), UNS), (dict(T=1 << 31), UNS),
])
def test_rope_refuses(bad, status):
    assert rope(**bad) == status
    assert lib.dsa_launch_count() == 0


def test_rope_freqs_refuses():
    f = (ctypes.c_double * 64)()
    at = ctypes.cast(f, P)
    good = [64, 1e4, 3, 8.0, 4096.0, 32.0, 1.0, at, None]
    assert lib.dsa_rope_freqs(*good) == dsa.DSA_OK and f[0] == 1.0
    for i, v in ((0, 0), (0, 63), (1, 1.0), (1, NAN), (2, 4), (2, -1), (3, 0.5), (3, NAN), (4, 0.0), (5, 1.0), (6, 0.0),
                 (7, None)):
        args = list(good)
        args[i] = v
        assert lib.dsa_rope_freqs(*args) == INV, (i, v)
    assert lib.dsa_rope_freqs(2, 1e4, 2, 8.0, 0.0, 0.0, 0.0, at, None) == INV
    with pytest.raises(ValueError):
        dsa.rope_freqs(64, scaling="cubic")
    with pytest.raises(dsa.DSAError):
        dsa.rope_freqs(-2)


def test_rope_freqs_formulas():
    f, m = dsa.rope_freqs(64, 1e4)
    assert m == 1.0 and np.allclose(f.numpy(), 1e4 ** (-np.arange(32) / 32), rtol=1e-14)
    lin, m = dsa.rope_freqs(64, 1e4, "linear", 8.0)
    assert m == 1.0 and np.allclose(lin.numpy(), f.numpy() / 8, rtol=1e-14)
    ntk, m = dsa.rope_freqs(64, 1e4, "ntk", 8.0)
    assert m == 1.0 and ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 8, rtol=1e-12)
    yarn, m = dsa.rope_freqs(64, 1e4, "yarn", 8.0, 4096)
    turns = 4096 * f.numpy() / (2 * np.pi)
    ratio = yarn.numpy() / f.numpy()
    assert np.isclose(m, 0.1 * np.log(8.0) + 1, rtol=1e-6)
    assert np.allclose(ratio[turns > 33 * 1.4], 1.0) and np.allclose(ratio[turns < 0.7], 1 / 8)
    assert np.all(np.diff(ratio) <= 1e-15)


def append(k=A, v=A, kts=512, khs=128, vts=512, vhs=128, N=3, cu=None, ctx=A, rpos=None, inv=A, off=0, R=64, layout=0,
           m=1.0, fmt=0, kp=A, vp=A, ks=A, vs=A, table=A, B=3, pages=9, page=64, most=3, Hkv=4, D=128):
    return lib.dsa_kv_append(k, v, kts, khs, vts, vhs, N, cu, ctx, rpos, inv, off, R, layout, m, fmt, kp, vp, ks, vs,
                             table, B, pages, page, most, Hkv, D, None)


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), INV), (dict(v=M), INV), (dict(ctx=None), INV), (dict(ctx=ODD), INV), (dict(cu=ODD), INV),
    (dict(rpos=ODD), INV), (dict(kp=None), INV), (dict(vp=M), INV), (dict(ks=None), INV), (dict(vs=ODD), INV),
    (dict(table=None), INV), (dict(N=0), INV), (dict(B=0), INV), (dict(N=4), INV), (dict(pages=0), INV),
    (dict(most=0), INV), (dict(kts=-8), INV), (dict(vhs=132), INV), (dict(fmt=2), INV), (dict(R=-16), INV),
    (dict(inv=None), INV), (dict(inv=M), INV), (dict(layout=3), INV), (dict(off=80), INV), (dict(m=NAN), INV),
    (dict(R=40), UNS), (dict(off=4), UNS), (dict(D=64, R=0), UNS), (dict(Hkv=3), UNS), (dict(Hkv=8), UNS),
    (dict(page=48), UNS), (dict(page=8), UNS), (dict(page=256), UNS), (dict(N=1 << 30, cu=A), UNS),
    (dict(most=1 << 25), UNS),
])
def test_append_refuses(bad, status):
    assert append(**bad) == status
    assert lib.dsa_launch_count() == 0


def attn(q=A, kp=A, vp=A, ks=A, vs=A, table=A, seq=None, n=A, idx=None, fmt=0, T=3, B=3, pages=9, page=64, most=3, Hq=32,
         Hkv=4, D=128, topk=0, scale=0.1, out=A, lse=None, ws=A, ws_bytes=1 << 30):
    return lib.dsa_paged_attn(q, kp, vp, ks, vs, table, seq, n, idx, fmt, T, B, pages, page, most, Hq, Hkv, D, topk, scale,
                              out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(q=M), INV), (dict(kp=None), INV), (dict(vp=M), INV), (dict(ks=ODD), INV),
    (dict(vs=None), INV), (dict(table=None), INV), (dict(n=None), INV), (dict(seq=ODD), INV), (dict(idx=ODD, topk=4), INV),
    (dict(lse=ODD), INV), (dict(out=None), INV), (dict(T=0), INV), (dict(T=4), INV), (dict(B=0, seq=A), INV),
    (dict(idx=A, topk=0), INV), (dict(fmt=-1), INV), (dict(scale=NAN), INV), (dict(pages=0), INV), (dict(most=-1), INV),
    (dict(Hq=0), INV), (dict(D=64), UNS), (dict(Hkv=3, Hq=24), UNS), (dict(Hq=30), UNS), (dict(Hq=68), UNS),
    (dict(page=24), UNS), (dict(idx=A, topk=65537), UNS), (dict(most=1 << 25), UNS),
    (dict(ws=None), WS), (dict(ws=M), WS), (dict(ws_bytes=1000), WS),
])
def test_attn_refuses(bad, status):
    assert attn(**bad) == status
    assert lib.dsa_launch_count() == 0


def _cache(B=2, pages=5, page=16, Hkv=2, fmt=torch.int8):
    z = torch.zeros
    return dict(k_pages=z((pages, page, Hkv, 128), dtype=torch.uint8).view(fmt),
                v_pages=z((pages, page, Hkv, 128), dtype=torch.uint8).view(fmt), k_scale=z(pages, Hkv),
                v_scale=z(pages, Hkv), page_table=z((B, 2), dtype=torch.int32))


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


CASES = [
    (dsa.dsa_rope, dict(x=_bf(4, 2, 64), out=_bf(4, 2, 64), inv_freq=torch.zeros(16, dtype=torch.float64), pos=_i32(4)),
     {"out": _bf(4, 2, 32), "inv_freq": torch.zeros(4, 4, dtype=torch.float64), "pos": _i32(5)},
     {"x": torch.zeros(4, 2, 64, dtype=torch.float16), "out": torch.zeros(4, 2, 64), "inv_freq": torch.zeros(16),
      "pos": torch.zeros(4, dtype=torch.int64)}),
    (dsa.dsa_kv_append, dict(k_new=_bf(6, 2, 128), v_new=_bf(6, 2, 128), **_cache(), ctx_len=_i32(2), cu_new=_i32(3),
                             inv_freq=torch.zeros(16, dtype=torch.float64), rope_pos=_i32(6)),
     {"k_new": _bf(6, 1, 128), "v_new": _bf(5, 2, 128), "v_pages": torch.zeros((5, 16, 1, 128), dtype=torch.int8),
      "k_scale": torch.zeros(4, 2), "v_scale": torch.zeros(5, 1), "page_table": _i32(2), "ctx_len": _i32(3),
      "cu_new": _i32(2), "rope_pos": _i32(2)},
     {"k_new": torch.zeros(6, 2, 128), "k_pages": torch.zeros((5, 16, 2, 128), dtype=torch.uint8),
      "v_pages": torch.zeros((5, 16, 2, 128), dtype=torch.uint8).view(torch.float8_e4m3fn), "k_scale": _bf(5, 2),
      "cu_new": torch.zeros(3, dtype=torch.int64)}),
    (dsa.dsa_paged_attn, dict(q=_bf(3, 8, 128), **_cache(fmt=torch.float8_e4m3fn), n_keys=_i32(3), scale=0.1,
                              out=_bf(3, 8, 128), seq=_i32(3), idx=_i32(3, 7), lse=torch.zeros(3, 8)),
     {"q": _bf(3, 8, 64), "n_keys": _i32(4), "out": _bf(3, 4, 128), "seq": _i32(2), "idx": _i32(2, 7),
      "lse": torch.zeros(3, 4)},
     {"q": torch.zeros(3, 8, 128), "n_keys": torch.zeros(3, dtype=torch.int64), "lse": _bf(3, 8)}),
]


@pytest.mark.parametrize("fn,args,shapes,types", CASES, ids=[c[0].__name__ for c in CASES])
def test_binding_checks_every_operand(fn, args, shapes, types):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn(**args)
    for name, wrong in shapes.items():
        with pytest.raises(ValueError, match=f"^{name}"):
            fn(**{**args, name: wrong})
    for name, wrong in types.items():
        with pytest.raises(TypeError, match=f"^{name}"):
            fn(**{**args, name: wrong})
    for name, t in args.items():
        if isinstance(t, torch.Tensor) and t.dim() == 2 and t.shape[1] > 1:
            with pytest.raises(ValueError, match=f"^{name}"):
                fn(**{**args, name: t.t().contiguous().t()})      # a transposed operand of the right shape


def test_binding_needs_a_sequence_for_every_row():
    (_, a, _, _), (_, b, _, _) = CASES[1], CASES[2]
    with pytest.raises(ValueError, match="^k_new"):
        dsa.dsa_kv_append(**{**a, "cu_new": None})
    with pytest.raises(ValueError, match="^q "):
        dsa.dsa_paged_attn(**{**b, "seq": None})
    with pytest.raises(ValueError, match="last axis"):
        dsa.dsa_rope(**{**CASES[0][1], "x": _bf(4, 64, 2).transpose(1, 2)})


def test_workspace_size_of_paged_attention_depends_on_heads_alone():
    w = [dsa.workspace_size(dsa.DSA_OP_PAGED_ATTN, L, B, 32, 1, 1) for L, B in ((1, 1), (1 << 20, 4096))]
    assert w[0] == w[1] > 0
    assert dsa.workspace_size(dsa.DSA_OP_PAGED_ATTN, 1, 1, 64, 1, 1) > w[0]
    assert dsa.workspace_size(dsa.DSA_OP_PAGED_ATTN, 1, 0, 32, 1, 1) == 0
