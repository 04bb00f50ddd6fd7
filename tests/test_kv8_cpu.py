"""The 8-bit cache and the NVFP4 linear layer without a device: refused
arguments (the binding's and the C ABI's, before any launch), workspace
sizes, and the 64-bit forms themselves."""
import ctypes as C

import pytest
import torch

import kv8_ref as ref
from bit_quantization_b200 import build, ops

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


def _cache(B=2, Hkv=2, cap=40, d=64, blk=16):
    k, v = (torch.zeros((B, Hkv, cap, d), dtype=torch.uint8).view(F8) for _ in range(2))
    ks, vs = (torch.zeros((B, Hkv, -(-cap // blk))) for _ in range(2))
    return k, v, ks, vs


N = torch.zeros(2, dtype=torch.int32)


def test_binding_refuses():
    k, v, ks, vs = _cache()
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    new = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)

    def decode(q=q, k=k, v=v, ks=ks, vs=vs, n=N, **kw):
        ops.thrift_kv8_decode(q, k, v, ks, vs, n, **{"blk": 16, **kw})

    def append(kn=new, vn=new, k=k, v=v, ks=ks, vs=vs, n=N, **kw):
        ops.thrift_kv8_append(kn, vn, k, v, ks, vs, n, **{"blk": 16, **kw})

    bad = [
        lambda: decode(),                                    # no CUDA device
        lambda: append(),
        lambda: decode(k=k.view(torch.uint8)),               # codes of another type
        lambda: decode(v=v[:, :, :39]),                      # shapes that differ
        lambda: decode(k=k.transpose(2, 3), v=v.transpose(2, 3)),
        lambda: decode(v=v.transpose(0, 1).contiguous().transpose(0, 1)),  # layouts that differ
        lambda: decode(blk=24),
        lambda: decode(blk=32),                              # scales of another block size
        lambda: decode(ks=ks.double()),
        lambda: decode(ks=ks[..., :1].expand(2, 2, 3)),
        lambda: decode(q=q[:, :3]),                          # 3 heads over 2
        lambda: decode(q=q[:1]),
        lambda: decode(q=q.float()),
        lambda: decode(n=N.long()),
        lambda: decode(n=N[:1]),
        lambda: decode(weight=torch.zeros(2, 2, 39)),
        lambda: decode(out=torch.zeros(2, 4, 64)),
        lambda: decode(lse=torch.zeros(4, 2)),
        lambda: append(kn=new[:, :2]),
        lambda: append(kn=new.half()),
        lambda: append(kn=new[..., :32], vn=new[..., :32]),
        lambda: append(n_new=N[:1]),
        lambda: append(new_len=N.long()),
        lambda: append(weight=torch.zeros(2, 2, 41)),
        lambda: ops.thrift_kv8_evict(k, v, ks, vs, torch.zeros(2, 2, 40), N, 0, *_cache(),
                                     torch.zeros(2, 2, 40), N.clone(), blk=16),
        lambda: ops.thrift_kv8_evict(k, v, ks, vs, torch.zeros(2, 2, 40), N, 8, *_cache(),
                                     torch.zeros(2, 2, 40), N.clone(), blk=16, sink=5, recent=4),
        lambda: ops.thrift_kv8_evict(k, v, ks, vs, torch.zeros(2, 2, 40), N, 20,
                                     *_cache(cap=19), torch.zeros(2, 2, 19), N.clone(), blk=16),
        lambda: ops.thrift_kv8_evict(k, v, ks, vs, torch.zeros(2, 2, 40), N, 20,
                                     *_cache(Hkv=1), torch.zeros(2, 1, 40), N.clone(), blk=16),
        lambda: ops.KV8Cache(1, 1, 0, device="cpu"),
        lambda: ops.KV8Cache(1, 1, 8, d=96, device="cpu"),
        lambda: ops.KV8Cache(1, 1, 8, blk=8, device="cpu"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ops.ThriftError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_linear_binding_refuses():
    x = torch.zeros((2, 64), dtype=torch.float16)
    codes, scales = torch.zeros((5, 32), dtype=torch.uint8), torch.zeros((5, 4), dtype=torch.uint8)
    g = torch.ones(1)
    for call in (
        lambda: ops.nvfp4_linear(x, codes, scales, g),  # no CUDA device
        lambda: ops.nvfp4_linear(x.float(), codes, scales, g),
        lambda: ops.nvfp4_linear(x[:, :48], codes[:, :24], scales[:, :3], g),  # K % 32
        lambda: ops.nvfp4_linear(x.expand(33, 2, 64).reshape(66, 64), codes, scales, g),
        lambda: ops.nvfp4_linear(x, codes[:, :16], scales, g),
        lambda: ops.nvfp4_linear(x, codes, scales[:4], g),
        lambda: ops.nvfp4_linear(x, codes, scales, g.double()),
        lambda: ops.nvfp4_linear(x, codes, scales, g, out=torch.zeros((2, 5))),
        lambda: ops.nvfp4_linear(x[0], codes, scales, g),
    ):
        with pytest.raises(ops.ThriftError):
            call()


P = C.c_void_p


def _decode(L, **kw):
    a = dict(q=P(1 << 20), dt=1, B=2, H=4, Hkv=2, d=64, blk=16, cap=40, sb=5120, sh=2560, st=64,
             k=P(1 << 21), v=P(1 << 22), ks=P(1 << 23), vs=P(1 << 24), n=P(1 << 25),
             scale=C.c_float(0.1), w=None, out=P(1 << 26), lse=P(1 << 27), ws=P(1 << 28),
             wb=1 << 40, stream=None)
    return L.thrift_kv8_decode(*{**a, **kw}.values())


def test_decode_abi_refuses(L):
    for kw, want in (
        (dict(dt=2), ops.ERR_ARG), (dict(B=0), ops.ERR_ARG), (dict(H=3), ops.ERR_ARG),
        (dict(Hkv=0), ops.ERR_ARG), (dict(H=0), ops.ERR_ARG), (dict(cap=0), ops.ERR_ARG),
        (dict(d=96), ops.ERR_UNSUPPORTED), (dict(blk=24), ops.ERR_UNSUPPORTED),
        (dict(B=65536), ops.ERR_UNSUPPORTED), (dict(cap=(1 << 30) + 1), ops.ERR_UNSUPPORTED),
        (dict(st=48), ops.ERR_ARG), (dict(st=72), ops.ERR_ARG), (dict(sh=2544), ops.ERR_ARG),
        (dict(sb=0), ops.ERR_ARG), (dict(sb=-5120), ops.ERR_ARG),
        (dict(scale=C.c_float(float("nan"))), ops.ERR_ARG),
        (dict(scale=C.c_float(float("inf"))), ops.ERR_ARG),
        (dict(q=None), ops.ERR_ARG), (dict(k=None), ops.ERR_ARG), (dict(v=None), ops.ERR_ARG),
        (dict(ks=None), ops.ERR_ARG), (dict(vs=None), ops.ERR_ARG), (dict(n=None), ops.ERR_ARG),
        (dict(out=None), ops.ERR_ARG), (dict(lse=None), ops.ERR_ARG), (dict(ws=None), ops.ERR_ARG),
        (dict(q=P(8)), ops.ERR_ARG), (dict(k=P(24)), ops.ERR_ARG), (dict(ws=P(8)), ops.ERR_ARG),
        (dict(wb=16), ops.ERR_ARG),
    ):
        assert _decode(L, **kw) == want, kw


def _append(L, **kw):
    a = dict(kn=P(1 << 20), vn=P(1 << 21), dt=1, B=2, Hkv=2, d=64, blk=16, cap=40, sb=5120,
             sh=2560, st=64, n=P(1 << 25), nn=None, T=3, k=P(1 << 22), v=P(1 << 23),
             ks=P(1 << 24), vs=P(1 << 25), w=None, nl=None, stream=None)
    return L.thrift_kv8_append(*{**a, **kw}.values())


def test_append_abi_refuses(L):
    for kw, want in (
        (dict(dt=-1), ops.ERR_ARG), (dict(T=-1), ops.ERR_ARG), (dict(kn=None), ops.ERR_ARG),
        (dict(vn=P(2)), ops.ERR_ARG), (dict(n=None), ops.ERR_ARG), (dict(v=P(1 << 22)), ops.ERR_ARG),
        (dict(blk=256), ops.ERR_UNSUPPORTED), (dict(sh=100), ops.ERR_ARG),
        (dict(ks=None), ops.ERR_ARG), (dict(T=0, kn=None, vn=None), ops.OK),  # launches nothing
    ):
        assert _append(L, **kw) == want, kw


def _evict(L, **kw):
    a = dict(B=2, Hkv=2, d=64, blk=16, cap=40, sb=5120, sh=2560, st=64, k=P(1 << 20), v=P(1 << 21),
             ks=P(1 << 22), vs=P(1 << 23), w=P(1 << 24), n=P(1 << 25), budget=20, sink=2, recent=3,
             cap_o=20, sbo=2560, sho=1280, sto=64, ko=P(1 << 26), vo=P(1 << 27), kso=P(1 << 28),
             vso=P(1 << 29), wo=P(1 << 30), lo=P(1 << 31), ws=P(1 << 32), wb=1 << 40, stream=None)
    return L.thrift_kv8_evict(*{**a, **kw}.values())


def test_evict_abi_refuses(L):
    for kw, want in (
        (dict(budget=0), ops.ERR_ARG), (dict(sink=-1), ops.ERR_ARG), (dict(recent=19), ops.ERR_ARG),
        (dict(cap_o=19), ops.ERR_ARG), (dict(budget=40, cap_o=39), ops.ERR_ARG),
        (dict(ko=P(1 << 20)), ops.ERR_ARG), (dict(ko=P((1 << 20) + 10224)), ops.ERR_ARG),
        (dict(wo=P(1 << 24)), ops.ERR_ARG), (dict(lo=P(1 << 25)), ops.ERR_ARG),
        (dict(vo=P(1 << 26)), ops.ERR_ARG), (dict(w=None), ops.ERR_ARG), (dict(wb=100), ops.ERR_ARG),
        (dict(sto=32), ops.ERR_ARG), (dict(d=32), ops.ERR_UNSUPPORTED),
        (dict(ws=P(1 << 30)), ops.ERR_ARG), (dict(st=1 << 24, sh=1 << 30, sb=1 << 31), ops.ERR_ARG),
    ):
        assert _evict(L, **kw) == want, kw


def test_linear_abi_refuses(L):
    def call(M=1, N=5, K=64, dt=0, x=P(1 << 20), c=P(1 << 21), s=P(1 << 22), g=P(1 << 23),
             out=P(1 << 24), ws=P(1 << 25), wb=1 << 40):
        return L.nvfp4_linear(x, dt, M, N, K, c, s, g, out, ws, wb, None)

    for kw, want in (
        (dict(dt=5), ops.ERR_ARG), (dict(M=-1), ops.ERR_ARG), (dict(K=24), ops.ERR_ARG),
        (dict(K=48), ops.ERR_UNSUPPORTED), (dict(M=65), ops.ERR_UNSUPPORTED),
        (dict(x=None), ops.ERR_ARG), (dict(c=P(8)), ops.ERR_ARG), (dict(g=None), ops.ERR_ARG),
        (dict(K=(1 << 19) + 32), ops.ERR_UNSUPPORTED), (dict(wb=16), ops.ERR_ARG), (dict(M=0), ops.OK), (dict(N=0), ops.OK),
    ):
        assert call(**kw) == want, kw


def test_workspace_sizes(L):
    assert L.thrift_kv8_decode_workspace_size(1, 1, 1, 1, 64, 0) > 0
    assert L.thrift_kv8_decode_workspace_size(1, 3, 2, 1, 64, 0) == 0
    assert L.thrift_kv8_decode_workspace_size(1, 1, 1, 1, 96, 0) == 0
    assert L.thrift_kv8_evict_workspace_size(2, 3, 100, 50) >= 2 * 3 * 50 * 4
    assert L.thrift_kv8_evict_workspace_size(2, 3, 100, 1 << 30) < 1 << 16
    assert L.nvfp4_linear_workspace_size(1, 10, 64) > 0
    assert L.nvfp4_linear_workspace_size(1, 10, 48) == 0
    assert L.nvfp4_linear_workspace_size(65, 10, 64) == 0


def test_reference_rounding_matches_the_type():
    """The reference's E4M3 rounding by spacing equals torch's conversion, and
    a power-of-two scale is minimal."""
    x = torch.cat([torch.linspace(-448, 448, 5001), torch.linspace(-0.1, 0.1, 5001),
                   torch.exp2(torch.arange(-12.0, 9.0))]).double()
    assert torch.equal(ref.e4m3(x), x.float().to(F8).view(torch.uint8))
    for a in (448.0, 448.1, 447.9, 1.0, 1e-30, 3e38, 0.875, 0.8750001):
        s = ref.scale_of(torch.tensor([a, -a / 2], dtype=torch.float64))
        assert a <= 448 * s and a > 448 * s / 2
    assert ref.scale_of(torch.tensor([0.0, float("inf"), float("nan")])) == 2.0 ** -120


def test_reference_rescale_is_exact_above_the_subnormals():
    """Moving codes to a larger power-of-two scale and back loses nothing that
    stays a normal E4M3 number."""
    code = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    code = code[(code & 0x7F) < 0x7F]
    v = ref.value(code)
    for shift in (1, 3, 8):
        keep = v.abs() >= 2.0 ** (-6 + shift)
        moved = ref.e4m3(v / 2.0 ** shift)
        assert torch.equal(ref.value(moved)[keep] * 2.0 ** shift, v[keep])
