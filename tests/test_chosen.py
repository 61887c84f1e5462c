"""Operators whose weights are chosen for each token: expert routing, the mixture-of-experts layer
on AWQ experts, and per-request low-rank adapters.

Tolerances, from the arithmetic (u = half a step of the output type, ``torch.finfo(t).eps / 2``):

* outputs are sums held in 32 bits and rounded once, so a row of the output is off by at most u of
  itself (each element's rounding), plus what the sums and their operands lose:
  - expert layer: x and h enter as 15-bit fixed point, 64 values to a scale of max / 16256: a value is
    off by at most half a step, max * 2^-15, with an rms of max * 2^-14 / sqrt(12). The largest of 64
    values is at most 8 times their rms, so a block is off by at most 8 * 2^-14 / sqrt(12) = 1.4e-4
    of its rms; x enters gate and up, h the output: 3 * 1.4e-4 < 2^-11 = EXTRA, the 32-bit sums
    (some 2^-20) included.
  - adapters: v enters as the sum of two 16-bit numbers, off by 2^-17 (bf16) of itself; two 32-bit sums
    of up to a few thousand terms add some 2^-20 each: 2^-15 with room.
* routing weights: exp(l - m) with |l - m| <= 32 is off by 32 * 2^-24 from the difference's rounding
  and 2 * 2^-24 from expf; the sum and the quotient add at most 20 roundings: 54 * 2^-24 < 4e-6.
"""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16
EXTRA = 2.0 ** -11
gpu = pytest.mark.gpu


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_rows_close(out, ref, dtype, extra=None):
    """Each row within (u + extra) of the reference's norm; rows of zeros exactly zero."""
    out, ref = f64(out), np.asarray(ref)
    assert out.shape == ref.shape
    assert np.isfinite(out).all()
    err = np.linalg.norm(out - ref, axis=-1)
    bound = (u_of(dtype) + (EXTRA if extra is None else extra)) * np.linalg.norm(ref, axis=-1)
    assert (err <= bound).all(), f"rows {np.nonzero(err > bound)[0][:8]}: {err.max():.3g} over {bound.min():.3g}"


@pytest.fixture(scope="module")
def ck():
    from bit_quantized_linear_rotate_b200 import build
    build.build()
    from bit_quantized_linear_rotate_b200 import ck as _ck
    return _ck


@pytest.fixture
def on_gpu(ck):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield ck
    ck.device_error_check()


# ------------------------------------------------------------------- inputs

def experts(E, K, I, G, dtype, seed):
    """(gate_up, down): packed bytes, scales and zeros of E experts, on the CPU."""
    g = torch.Generator().manual_seed(seed)

    def part(rows, cols):
        return (torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8),
                (torch.rand((E, cols // G, rows), generator=g) * 0.009 + 0.001).to(dtype),
                (torch.randn((E, cols // G, rows), generator=g) * 0.01).to(dtype))

    return part(2 * I, K), part(K, I)


def to_dev(parts):
    return [t.to(DEV) for t in parts]


def moe_ref(x, ids, weights, gu, dn, G):
    return O.moe_awq_w4a16(f64(x), ids.cpu().numpy(), f64(weights), [gu[0].numpy(), f64(gu[1]), f64(gu[2])],
                           [dn[0].numpy(), f64(dn[1]), f64(dn[2])], G)


def adapters(M, K, N, R, L, dtype, ydtype, seed, runs=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).to(dtype)
    y = torch.randn((M, N), generator=g).to(ydtype)
    a = (torch.randn((L, R, K), generator=g) / K ** 0.5).to(dtype)
    b = (torch.randn((L, N, R), generator=g) / R ** 0.5).to(dtype)
    ids = torch.randint(-1, L, (-(-M // runs),), generator=g, dtype=torch.int32).repeat_interleave(runs)[:M]
    scales = torch.rand((L,), generator=g) + 0.5
    return x, y, a, b, ids.contiguous(), scales


def lora_ref(x, y, a, b, ids, scales):
    return O.lora_add(f64(y), f64(x), f64(a), f64(b), ids.cpu().numpy(), None if scales is None else f64(scales))


# ------------------------------------------------------- the oracle, on CPU

def test_oracle_route_by_hand():
    inf = np.inf
    w, ids = O.moe_route([[1.0, 3.0, 3.0, -inf], [-inf, np.nan, -inf, 0.0], [inf, 2.0, inf, inf], [np.nan] * 4], 2, True)
    assert ids.tolist() == [[1, 2], [3, -1], [0, 2], [-1, -1]]
    np.testing.assert_allclose(w, [[0.5, 0.5], [1.0, 0.0], [0.5, 0.5], [0.0, 0.0]])
    w, _ = O.moe_route([[0.0, np.log(2.0), np.log(5.0), -inf]], 2, False)
    np.testing.assert_allclose(w, [[5 / 8, 2 / 8]])


def test_oracle_moe_by_hand():
    # one expert whose weights are all (u - 8) s + z = 0.5: gate = up = 0.5 sum(x), out = 0.5 I h
    K = I = 64
    gu = (np.full((1, 2 * I, K // 2), 0x99), np.full((1, 1, 2 * I), 0.25), np.full((1, 1, 2 * I), 0.25))
    dn = (np.full((1, K, I // 2), 0x99), np.full((1, 1, K), 0.25), np.full((1, 1, K), 0.25))
    x = np.full((2, K), 1 / 16)
    out = O.moe_awq_w4a16(x, np.array([[0, 0], [-1, 7]]), np.array([[1.0, 0.5], [1.0, 1.0]]), gu, dn, 64)
    v = 2.0
    np.testing.assert_allclose(out[0], 1.5 * 32 * (v / (1 + np.exp(-v)) * v))
    assert not out[1].any()


def test_oracle_lora_by_hand():
    out = O.lora_add([[1.0, 2.0]], [[1.0, 1.0]], [[[1.0, 2.0]]], [[[10.0], [20.0]]], [0], [0.5])
    np.testing.assert_allclose(out, [[1 + 15.0, 2 + 30.0]])
    np.testing.assert_allclose(O.lora_add([[1.0]], [[1.0]], [[[1.0]]], [[[1.0]]], [1]), [[1.0]])


# ----------------------------------------------------------- refusals, CPU

P = ctypes.c_void_p


def route_call(ck, **kw):
    a = dict(logits=P(1 << 20), lt=2, T=4, E=8, k=2, w=P(1 << 21), ids=P(1 << 22))
    a.update(kw)
    return ck.lib.ck_moe_route(a["logits"], a["lt"], a["T"], a["E"], a["k"], 1, a["w"], a["ids"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(E=513), 2), (dict(E=64, k=17), 2),
    (dict(lt=3), 1), (dict(logits=None), 1), (dict(w=None), 1), (dict(ids=None), 1), (dict(logits=P((1 << 20) + 2)), 1),
    (dict(w=P((1 << 21) + 2)), 1), (dict(T=1 << 40), 2), (dict(T=0, logits=None, w=None, ids=None), 0)])
def test_route_validation(ck, kw, status):
    assert route_call(ck, **kw) == status
    assert (ck.last_error() == "") == (status == 0)


def moe_call(ck, given=False, **kw):
    p = P(1 << 20)
    a = dict(x=p, dt=0, T=4, K=128, I=64, E=8, ldx=128, G=64, logits=p, lt=2, k=2, gq=p, gs=p, gz=p, dq=p, ds=p, dz=p,
             out=p, ws=P(1 << 21), bytes=None, ids=p, w=p)
    a.update(kw)
    n = ck.moe_awq_w4a16_workspace_bytes(a["T"], a["k"], a["K"], a["I"]) if a["bytes"] is None else a["bytes"]
    head = (a["x"], a["dt"], a["T"], a["K"], a["I"], a["E"], a["ldx"], a["G"])
    tail = (a["gq"], a["gs"], a["gz"], a["dq"], a["ds"], a["dz"], a["out"], a["ws"], n, None)
    if given:
        return ck.lib.ck_moe_experts_awq_w4a16(*head, a["ids"], a["w"], a["k"], *tail)
    return ck.lib.ck_moe_awq_w4a16(*head, a["logits"], a["lt"], a["k"], 1, *tail)


off = P((1 << 20) + 8)


@pytest.mark.parametrize("kw,status", [
    (dict(T=65), 2), (dict(T=-1), 1), (dict(K=0), 1), (dict(I=0), 1), (dict(E=0), 1), (dict(E=513), 2), (dict(k=0), 1),
    (dict(E=64, k=17), 2), (dict(dt=2), 1), (dict(G=32), 2), (dict(G=192, K=192, I=192, ldx=192), 2), (dict(G=0), 2),
    (dict(K=96, ldx=96), 1), (dict(I=96), 1), (dict(G=128), 1), (dict(ldx=64), 1), (dict(ldx=132), 1),
    (dict(K=1 << 21, ldx=1 << 21), 2), (dict(x=None), 1), (dict(gq=None), 1), (dict(gs=None), 1), (dict(gz=None), 1),
    (dict(dq=None), 1), (dict(ds=None), 1), (dict(dz=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(x=off), 1), (dict(gq=off), 1), (dict(gs=off), 1), (dict(gz=off), 1), (dict(dq=off), 1), (dict(ds=off), 1),
    (dict(dz=off), 1), (dict(out=P((1 << 20) + 1)), 1), (dict(ws=P((1 << 21) + 128)), 1), (dict(bytes=100), 1),
    (dict(T=0, x=None, logits=None, ids=None, w=None, out=None, ws=None), 0)])
@pytest.mark.parametrize("given", [False, True])
def test_moe_validation(ck, given, kw, status):
    assert moe_call(ck, given, **kw) == status
    assert (ck.last_error() == "") == (status == 0)


def test_moe_choice_validation(ck):
    assert moe_call(ck, logits=None) == 1
    assert moe_call(ck, lt=3) == 1
    assert moe_call(ck, k=9) == 1                           # more than there are experts
    assert moe_call(ck, True, ids=None) == 1
    assert moe_call(ck, True, w=None) == 1
    assert moe_call(ck, True, w=P((1 << 20) + 2)) == 1
    # x and h in records of 576 bytes for 256 columns, the lists: each rounded up to 256 bytes
    assert ck.moe_awq_w4a16_workspace_bytes(4, 2, 320, 64) == 18 * 256 + 18 * 256 + 256
    assert ck.moe_awq_w4a16_workspace_bytes(0, 2, 128, 64) == 0


def lora_call(ck, **kw):
    a = dict(y=P(1 << 20), yt=0, x=P(1 << 24), xt=0, M=4, K=64, N=40, R=16, L=3, ldx=64, ldy=40, ldo=40, a=P(1 << 25),
             b=P(1 << 25), ids=P(1 << 25), s=P(1 << 25), out=P(1 << 20), ws=None, bytes=0)
    a.update(kw)
    return ck.lib.ck_lora_add(a["y"], a["yt"], a["x"], a["xt"], a["M"], a["K"], a["N"], a["R"], a["L"], a["ldx"],
                              a["ldy"], a["ldo"], a["a"], a["b"], a["ids"], a["s"], a["out"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(R=0), 1), (dict(L=0), 1), (dict(xt=2), 1), (dict(yt=2), 1),
    (dict(yt=1), 2), (dict(R=12), 2), (dict(R=136), 2), (dict(K=60), 2), (dict(L=8193), 2), (dict(M=(1 << 26) + 1), 2),
    (dict(N=1 << 31), 2), (dict(N=1 << 28, L=8), 2), (dict(ldx=56), 1), (dict(ldx=68), 1), (dict(ldy=39), 1), (dict(ldo=39), 1),
    (dict(y=None), 1), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ids=None), 1), (dict(out=None), 1),
    (dict(x=P((1 << 24) + 8)), 1), (dict(a=P((1 << 25) + 8)), 1), (dict(b=P((1 << 25) + 8)), 1),
    (dict(ids=P((1 << 25) + 2)), 1), (dict(s=P((1 << 25) + 2)), 1), (dict(out=P((1 << 20) + 1)), 1),
    (dict(out=P((1 << 20) + 16)), 1),                      # overlaps y without being y
    (dict(ldo=48), 1), (dict(out=P((1 << 24) + 16)), 1),   # over x
    (dict(M=257, L=2000), 1), (dict(M=257, L=2000, ws=P(1 << 26), bytes=64), 1),
    (dict(M=257, L=2000, ws=P((1 << 26) + 16), bytes=1 << 20), 1),
    (dict(M=0, y=None, x=None, a=None, b=None, ids=None, out=None), 0)])
def test_lora_validation(ck, kw, status):
    assert lora_call(ck, **kw) == status
    assert (ck.last_error() == "") == (status == 0)


def test_lora_workspace_bytes(ck):
    for M, L in ((1, 1), (256, 8192), (257, 1), (257, 9), (777, 5), (4096, 1024), (32768, 1024)):
        assert ck.lora_add_workspace_bytes(M, L) == 0       # every CTA finds its tile itself
    for M, L in ((4097, 1024), (32769, 1), (32768, 1025), (257, 1025), (300, 8192)):
        n = ck.lora_add_workspace_bytes(M, L)
        assert n >= 4 * M + 16 * (M // 128 + min(L, 1))     # the token order, and 16 bytes a tile


def test_binding_refuses_shapes_and_dtypes_before_any_launch(ck):
    x = torch.zeros(4, 128, dtype=BF)
    gu, dn = experts(2, 128, 64, 64, BF, 0)
    logits = torch.zeros(4, 2)
    with pytest.raises(TypeError, match="logits"):
        ck.moe_route(logits.double(), 1)
    with pytest.raises(ValueError, match="logits"):
        ck.moe_route(torch.zeros(2, 4).t(), 1)
    with pytest.raises(ValueError, match="weights_out"):
        ck.moe_route(logits, 2, weights_out=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        ck.moe_route(logits, 1)
    with pytest.raises(TypeError, match="gate_up_s"):
        ck.moe_awq_w4a16(x, logits, 1, gu[0], gu[1].half(), gu[2], *dn)
    with pytest.raises(ValueError, match="down_q"):
        ck.moe_awq_w4a16(x, logits, 1, *gu, dn[0][:, :64], dn[1], dn[2])
    with pytest.raises(ValueError, match="logits"):
        ck.moe_awq_w4a16(x, torch.zeros(4, 3), 1, *gu, *dn)
    with pytest.raises(TypeError, match="ids"):
        ck.moe_experts_awq_w4a16(x, torch.zeros(4, 1, dtype=torch.int64), torch.zeros(4, 1), *gu, *dn)
    with pytest.raises(ValueError, match="weights"):
        ck.moe_experts_awq_w4a16(x, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 2), *gu, *dn)
    with pytest.raises(ValueError, match="CUDA"):
        ck.moe_awq_w4a16(x, logits, 1, *gu, *dn)
    x, y, a, b, ids, scales = adapters(4, 64, 40, 8, 3, BF, BF, 0)
    with pytest.raises(TypeError, match="lora_a"):
        ck.lora_add(y, x, a.half(), b, ids)
    with pytest.raises(TypeError, match="y"):
        ck.lora_add(y.half(), x, a, b, ids)
    with pytest.raises(TypeError, match="ids"):
        ck.lora_add(y, x, a, b, ids.long())
    with pytest.raises(ValueError, match="lora_b"):
        ck.lora_add(y, x, a, b[:, :, :4].contiguous(), ids)
    with pytest.raises(ValueError, match="y must be"):
        ck.lora_add(y[:3], x, a, b, ids)
    with pytest.raises(ValueError, match="y must be"):
        ck.lora_add(y.t().contiguous().t(), x, a, b, ids)    # columns are contiguous, rows are not
    with pytest.raises(ValueError, match="x must be"):
        ck.lora_add(y, x[0], a, b, ids)
    with pytest.raises(ValueError, match="scales"):
        ck.lora_add(y, x, a, b, ids, scales=torch.zeros(2))
    with pytest.raises(ValueError, match="ids"):
        ck.lora_add(y, x, a, b, ids[:3])
    with pytest.raises(TypeError, match="out"):
        ck.lora_add(y, x, a, b, ids, out=y.half())
    with pytest.raises(ValueError, match="CUDA"):
        ck.lora_add(y, x, a, b, ids, scales)


# ------------------------------------------------------------------ routing

@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF, FP])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 33, 7), (64, 128, 8), (5, 129, 16), (2, 512, 16), (301, 60, 6)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(on_gpu, T, E, k, dtype, renorm):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (torch.randn((T, E), generator=g) * 2).to(dtype)     # 16-bit logits tie often
    w, ids = on_gpu.moe_route(logits.to(DEV), k, renormalize=renorm)
    w_ref, ids_ref = O.moe_route(f64(logits), k, renorm)
    assert ids.dtype == torch.int32 and np.array_equal(ids.cpu().numpy(), ids_ref)
    np.testing.assert_allclose(f64(w), w_ref, rtol=4e-6, atol=0)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF, FP])
def test_route_special_values(on_gpu, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    rows = [[-inf] * 6, [nan] * 6, [nan, -inf, 1, nan, -inf, nan], [inf, 3, inf, -inf, nan, 1], [0.0, -0.0, 0.0, -0.0, -1, 1],
            [low, low, -inf, low, low, low], [low, 0, low, nan, low, low], [2, 2, 2, 2, 2, 2], [inf] * 6]
    logits = torch.tensor(rows, dtype=torch.float64).to(dtype)
    for renorm in (True, False):
        w, ids = on_gpu.moe_route(logits.to(DEV), 4, renormalize=renorm)
        w_ref, ids_ref = O.moe_route(f64(logits), 4, renorm)
        assert np.array_equal(ids.cpu().numpy(), ids_ref)
        np.testing.assert_allclose(f64(w), w_ref, rtol=4e-6, atol=1e-38)


@gpu
def test_route_empty_and_given_outputs(on_gpu):
    w, ids = on_gpu.moe_route(torch.zeros((0, 4), device=DEV), 2)
    assert w.shape == (0, 2) and ids.shape == (0, 2)
    logits = torch.randn((7, 16), device=DEV)
    wo, io = torch.empty((7, 3), device=DEV), torch.empty((7, 3), device=DEV, dtype=torch.int32)
    w, ids = on_gpu.moe_route(logits, 3, weights_out=wo, ids_out=io)
    assert w is wo and ids is io and (ids >= 0).all()


# ------------------------------------------------------- mixture of experts

@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,E,k,K,I,G", [
    (1, 1, 1, 64, 64, 64), (1, 4, 2, 128, 64, 64), (2, 8, 8, 192, 320, 64), (5, 20, 3, 1472, 704, 64),
    (8, 6, 2, 256, 1024, 128), (9, 5, 4, 512, 512, 256), (16, 64, 8, 256, 128, 64), (17, 3, 3, 128, 192, 64),
    (33, 300, 5, 64, 128, 64), (64, 8, 2, 384, 640, 128), (64, 512, 16, 64, 64, 64),
    (4, 20, 16, 64, 64, 64), (4, 5, 2, 5120, 64, 64), (2, 4, 2, 512, 256, 256), (4, 3, 2, 384, 128, 128),
    (3, 200, 10, 128, 320, 64), (12, 16, 4, 960, 1088, 64)])
def test_moe(on_gpu, T, E, k, K, I, G, dtype):
    gu, dn = experts(E, K, I, G, dtype, T + E)
    g = torch.Generator().manual_seed(7)
    x = torch.randn((T, K), generator=g).to(dtype)
    logits = torch.randn((T, E), generator=g)
    out = on_gpu.moe_awq_w4a16(x.to(DEV), logits.to(DEV), k, *to_dev(gu), *to_dev(dn), group_size=G)
    w, ids = O.moe_route(f64(logits), k, True)
    assert out.dtype == dtype
    assert_rows_close(out, moe_ref(x, torch.tensor(ids), torch.tensor(w), gu, dn, G), dtype)


@gpu
@pytest.mark.parametrize("T,E", [(1, 5), (4, 5), (8, 5), (12, 5), (16, 5), (20, 5), (32, 5), (40, 5), (64, 5), (64, 400),
                                 (40, 60), (7, 1)])
def test_moe_all_tokens_on_one_expert(on_gpu, T, E):
    # more tokens than one pass over an expert's weights takes, next to experts without any
    K, I = 128, 192
    gu, dn = experts(E, K, I, 64, BF, T)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, K), generator=g).to(BF)
    ids = torch.full((T, 1), min(3, E - 1), dtype=torch.int32)
    w = torch.rand((T, 1), generator=g) + 0.1
    out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *to_dev(gu), *to_dev(dn))
    assert_rows_close(out, moe_ref(x, ids, w, gu, dn, 64), BF)


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
def test_moe_given_choice_with_empty_and_repeated_slots(on_gpu, dtype):
    E, K, I, k = 6, 256, 128, 4
    gu, dn = experts(E, K, I, 64, dtype, 3)
    g = torch.Generator().manual_seed(3)
    ids = torch.tensor([[0, 1, 2, 3], [2, 2, 2, 2], [-1, -1, -1, -1], [5, -7, 5, 0], [6, 99, 1, 1 << 30], [4, 1, 4, 1]],
                       dtype=torch.int32)
    w = torch.randn((6, k), generator=g)                    # any weights, negative ones too
    w[4, 1] = float("nan")                                  # the weight of an empty slot counts for nothing
    x = torch.randn((6, K), generator=g).to(dtype)
    out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *to_dev(gu), *to_dev(dn))
    ref = moe_ref(x, ids, torch.nan_to_num(w), gu, dn, 64)
    assert_rows_close(out, ref, dtype)
    assert not out[2].any()


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
def test_moe_given_choice_of_few_tokens(on_gpu, dtype):
    # the same for one and two tokens, which route in every block, and for the lists of three and four
    E, K, I = 7, 320, 192
    gu, dn = experts(E, K, I, 64, dtype, 4)
    g = torch.Generator().manual_seed(4)
    for rows in ([[2, 2, 2, 2]], [[-1, -1, 9, -5]], [[6, 0, 6, 1], [1, 1, 0, -1]], [[0, 0, 0], [-1, -1, -1]],
                 [[4], [4]], [[1, 2, 3, 4, 5, 6, 0, 1, 1, 1], [6, 6, 0, 5, 4, 3, 2, 1, 0, 0]], [[6, 0, 6, 1], [1, 1, 0, -1], [-1, -1, -1, -1], [0, 6, 1, 1]],
                 [[3], [3], [3], [3]], [[1, 2, 3, 4, 5, 6, 0, 1, 1, 1]] * 3):
        ids = torch.tensor(rows, dtype=torch.int32)
        w = torch.randn(ids.shape, generator=g)
        x = torch.randn((ids.shape[0], K), generator=g).to(dtype)
        out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *to_dev(gu), *to_dev(dn))
        assert_rows_close(out, moe_ref(x, ids, w, gu, dn, 64), dtype)
        assert not out[(ids < 0).all(1).to(DEV)].any()


@gpu
@pytest.mark.parametrize("T", [1, 2, 4, 16])
def test_moe_equals_route_and_given_experts_bit_for_bit(on_gpu, T):
    E, k, K, I = 32, 6, 512, 256
    gu, dn = experts(E, K, I, 64, BF, 1)
    gu, dn = to_dev(gu), to_dev(dn)
    x, logits = torch.randn((T, K), device=DEV).to(BF), torch.randn((T, E), device=DEV).to(BF)
    for renorm in (True, False):
        w, ids = on_gpu.moe_route(logits, k, renormalize=renorm)
        a = on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn, renormalize=renorm)
        b = on_gpu.moe_experts_awq_w4a16(x, ids, w, *gu, *dn)
        assert torch.equal(a, b)
        assert torch.equal(a, on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn, renormalize=renorm))


@gpu
def test_moe_tokens_do_not_depend_on_their_neighbours(on_gpu):
    # a token's output is the same alone and in a batch to within the order of its sums, and a
    # token that is not finite leaves the others as they are
    T, E, k, K, I = 12, 8, 2, 256, 192
    gu, dn = experts(E, K, I, 64, BF, 5)
    gu, dn = to_dev(gu), to_dev(dn)
    x, logits = torch.randn((T, K), device=DEV).to(BF), torch.randn((T, E), device=DEV)
    out = on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn)
    for t in (0, 7, 11):
        one = on_gpu.moe_awq_w4a16(x[t:t + 1], logits[t:t + 1], k, *gu, *dn)
        assert_rows_close(one, f64(out[t:t + 1]), BF, extra=u_of(BF) + EXTRA)
    bad = x.clone()
    bad[3, 17] = float("inf")
    bad[8, 200] = float("nan")
    got = on_gpu.moe_awq_w4a16(bad, logits, k, *gu, *dn)
    rest = [t for t in range(T) if t not in (3, 8)]
    assert torch.equal(got[rest], out[rest])
    assert not torch.isfinite(got[8]).any()
    masked = logits.clone()
    masked[5] = -float("inf")                               # a padded row: no expert
    got = on_gpu.moe_awq_w4a16(x, masked, k, *gu, *dn)
    assert not got[5].any()
    pair = on_gpu.moe_awq_w4a16(bad[2:4], logits[2:4], k, *gu, *dn)
    assert torch.equal(pair[0], on_gpu.moe_awq_w4a16(x[2:4], logits[2:4], k, *gu, *dn)[0])
    assert not torch.isfinite(pair[1]).any()
    pair = on_gpu.moe_awq_w4a16(x[4:6], masked[4:6], k, *gu, *dn)
    assert pair[0].any() and not pair[1].any()


@gpu
@pytest.mark.parametrize("T", [1, 2, 5, 40])
@pytest.mark.parametrize("K,I,G", [(192, 320, 64), (384, 128, 128), (256, 768, 256)])
def test_moe_experts_that_no_token_names_do_not_show(on_gpu, T, K, I, G):
    E = 5
    gu, dn = experts(E, K, I, G, BF, 21)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, K), generator=g).to(BF)
    ids = torch.tensor([[1, 3]] * T, dtype=torch.int32)
    w = torch.rand((T, 2), generator=g) + 0.1
    ref = moe_ref(x, ids, w, gu, dn, G)
    for i in (0, 2, 4):
        for t in (gu[1], gu[2], dn[1], dn[2]):
            t[i] = float("nan")
    out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *to_dev(gu), *to_dev(dn), group_size=G)
    assert_rows_close(out, ref, BF)


@gpu
def test_moe_strided_x_in_place_and_workspace_bounds(on_gpu):
    T, E, k, K, I = 10, 4, 2, 192, 128
    gu, dn = experts(E, K, I, 64, FP, 9)
    gu, dn = to_dev(gu), to_dev(dn)
    wide = torch.randn((T, K + 40), device=DEV).to(FP)
    logits = torch.randn((T, E), device=DEV)
    x = wide[:, 8:8 + K]
    ref = on_gpu.moe_awq_w4a16(x.contiguous(), logits, k, *gu, *dn)
    assert torch.equal(on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn), ref)
    need = on_gpu.moe_awq_w4a16_workspace_bytes(T, k, K, I)
    ws = torch.full((need + 256,), 0xA5, device=DEV, dtype=torch.uint8)
    buf = torch.full((T + 2, K), 7.0, device=DEV, dtype=FP)
    on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn, workspace=ws[:need], out=buf[1:-1])
    assert torch.equal(buf[1:-1], ref) and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert (ws[need:] == 0xA5).all()
    xc = x.contiguous()
    assert on_gpu.moe_awq_w4a16(xc, logits, k, *gu, *dn, out=xc) is xc
    assert torch.equal(xc, ref)
    empty = on_gpu.moe_awq_w4a16(x[:0], logits[:0], k, *gu, *dn)
    assert empty.shape == (0, K)
    with pytest.raises(on_gpu.CKError, match="T=65"):
        on_gpu.moe_awq_w4a16(torch.zeros((65, K), device=DEV, dtype=FP), torch.zeros((65, E), device=DEV), k, *gu, *dn)


@gpu
def test_moe_large_and_cancelling_h(on_gpu):
    # h far beyond fp16's range (1e6 and more) in an fp16 model, weights that bring it back
    T, E, K, I = 3, 2, 128, 64
    gu, dn = experts(E, K, I, 64, FP, 11)
    dn = (dn[0], (dn[1].float() * 1e-4).to(FP), (dn[2].float() * 1e-4).to(FP))
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((T, K), generator=g) * 4000).to(FP)
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32)
    w = torch.ones((T, 2)) * 1e-3
    out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *to_dev(gu), *to_dev(dn))
    ref = moe_ref(x, ids, w, gu, dn, 64)
    assert np.abs(ref).max() < 6e4
    assert_rows_close(out, ref, FP)


@gpu
def test_moe_graph_replay_streams_and_a_shared_workspace(on_gpu):
    T, E, k, K, I = 4, 16, 4, 256, 192
    gu, dn = experts(E, K, I, 64, BF, 13)
    gu, dn = to_dev(gu), to_dev(dn)
    x, logits = torch.randn((T, K), device=DEV).to(BF), torch.randn((T, E), device=DEV)
    ws = torch.empty(on_gpu.moe_awq_w4a16_workspace_bytes(T, k, K, I), device=DEV, dtype=torch.uint8)
    out, out2 = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    graphs = []
    for o in (out, out2):                                   # two graphs on one workspace, run in turn
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn, workspace=ws, out=o)
            on_gpu.moe_awq_w4a16(o, logits, k, *gu, *dn, workspace=ws, out=o)
        graphs.append(gr)
    for s in range(3):
        x.copy_(torch.randn((T, K), device=DEV).to(BF))
        logits.copy_(torch.randn((T, E), device=DEV))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        ref = on_gpu.moe_awq_w4a16(on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn), logits, k, *gu, *dn)
        assert torch.equal(out, ref) and torch.equal(out2, ref)
    torch.cuda.synchronize()
    got = on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn, stream=side)   # a stream that is not current
    side.synchronize()
    assert torch.equal(got, on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn))


# ----------------------------------------------------------------- adapters

@gpu
@pytest.mark.parametrize("dtype,ydtype", [(BF, BF), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("M,K,N,R,L,runs", [
    (1, 8, 1, 8, 1, 1), (1, 3840, 512, 16, 8, 1), (3, 64, 33, 8, 2, 1), (16, 256, 64, 24, 3, 2), (17, 264, 100, 32, 4, 1),
    (64, 512, 320, 40, 48, 1), (200, 136, 72, 64, 3, 70), (256, 128, 96, 128, 300, 1), (257, 128, 96, 72, 2, 50),
    (513, 200, 129, 16, 3, 100), (777, 1480, 1001, 24, 5, 150), (1030, 96, 256, 128, 4, 1), (600, 64, 64, 8, 2000, 1),
    (2100, 320, 200, 64, 7, 333), (300, 8, 40, 8, 1, 300), (1000, 64, 520, 48, 2, 1), (1500, 1000, 392, 112, 3, 400),
    (400, 200, 130, 56, 2, 64), (33000, 16, 24, 8, 2, 700), (9000, 24, 16, 16, 200, 3), (20000, 16, 40, 16, 300, 77),
    (4096, 16, 24, 8, 1000, 1), (4097, 8, 24, 8, 500, 2), (512, 136, 264, 16, 1, 1), (300, 64, 520, 96, 100, 1)])
def test_lora(on_gpu, M, K, N, R, L, runs, dtype, ydtype):
    x, y, a, b, ids, scales = adapters(M, K, N, R, L, dtype, ydtype, M + R, runs)
    args = [t.to(DEV) for t in (y, x, a, b, ids)]
    out = on_gpu.lora_add(*args, scales=scales.to(DEV))
    assert out.dtype == ydtype and torch.equal(args[0].cpu(), y)
    assert_rows_close(out, lora_ref(x, y, a, b, ids, scales), ydtype, extra=2.0 ** -15)
    none = (ids < 0).to(DEV)
    assert torch.equal(out[none], args[0][none])
    plain = on_gpu.lora_add(*args)
    assert_rows_close(plain, lora_ref(x, y, a, b, ids, None), ydtype, extra=2.0 ** -15)
    assert torch.equal(on_gpu.lora_add(*args, scales=scales.to(DEV)), out)         # the same bits again
    on_gpu.lora_add(*args, scales=scales.to(DEV), out=args[0])                      # in place
    assert torch.equal(args[0], out)


@gpu
def test_lora_ids_outside_the_adapters_and_strides(on_gpu):
    M, K, N, R, L = 300, 192, 120, 16, 4
    x, y, a, b, _, scales = adapters(M, K, N, R, L, BF, BF, 2)
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-3, L + 3, (M,), generator=g, dtype=torch.int32)
    ids[5], ids[6] = -(1 << 31), (1 << 31) - 1
    ref = lora_ref(x, y, a, b, ids, scales)
    wx, wy, wo = (torch.full((M, n + 24), 3.0, device=DEV, dtype=BF) for n in (K, N, N))
    wx[:, 8:8 + K], wy[:, 8:8 + N] = x.to(DEV), y.to(DEV)
    rest = [t.to(DEV) for t in (a, b, ids, scales)]
    for at in (8, 5):                                       # aligned rows, and rows that are not
        wy2 = torch.full((M, N + 24), 3.0, device=DEV, dtype=BF)
        wy2[:, at:at + N] = y.to(DEV)
        wo.fill_(3.0)
        got = on_gpu.lora_add(wy2[:, at:at + N], wx[:, 8:8 + K], *rest, out=wo[:, at:at + N])
        assert_rows_close(got, ref, BF, extra=2.0 ** -15)
        assert (wo[:, :at] == 3).all() and (wo[:, at + N:] == 3).all()
        on_gpu.lora_add(wy2[:, at:at + N], wx[:, 8:8 + K], *rest, out=wy2[:, at:at + N])
        assert torch.equal(wy2[:, at:at + N], got) and (wy2[:, :at] == 3).all() and (wy2[:, at + N:] == 3).all()
    with pytest.raises(on_gpu.CKError, match="overlaps"):
        on_gpu.lora_add(wy[:, 8:8 + N], wx[:, 8:8 + K], *rest, out=wy[:, 16:16 + N])


@gpu
@pytest.mark.parametrize("dtype,ydtype", [(BF, BF), (FP, BF)])
@pytest.mark.parametrize("N", [200, 264])
def test_lora_prompts_in_wider_matrices(on_gpu, N, dtype, ydtype):
    # consecutive tokens (tensor copies and stores): nothing outside the columns and rows is written, in place
    # or not, whatever the row strides; a tile ends at the last token
    M, K, R, L = 1000, 136, 24, 3
    x, y, a, b, _, scales = adapters(M, K, N, R, L, dtype, ydtype, 12)
    ids = torch.cat([torch.full((n,), i, dtype=torch.int32) for n, i in ((256, 2), (300, 0), (44, -1), (144, 1), (256, 0))])
    ref = lora_ref(x, y, a, b, ids, scales)
    wx = torch.full((M + 2, K + 24), 3.0, device=DEV, dtype=dtype)
    wy, wo = (torch.full((M + 2, N + 40), 3.0, device=DEV, dtype=ydtype) for _ in range(2))
    wx[1:-1, 8:8 + K], wy[1:-1, 16:16 + N] = x.to(DEV), y.to(DEV)
    rest = [t.to(DEV) for t in (a, b, ids, scales)]
    vx, vy, vo = wx[1:-1, 8:8 + K], wy[1:-1, 16:16 + N], wo[1:-1, 16:16 + N]
    on_gpu.lora_add(vy, vx, *rest, out=vo)
    assert_rows_close(vo, ref, ydtype, extra=2.0 ** -15)
    got = vo.clone()
    vo.fill_(3.0)
    assert (wo == 3).all()
    on_gpu.lora_add(vy, vx, *rest, out=vy)
    assert torch.equal(vy, got)
    assert (wy[0] == 3).all() and (wy[-1] == 3).all() and (wy[:, :16] == 3).all() and (wy[:, 16 + N:] == 3).all()


@gpu
def test_lora_rows_that_are_not_finite_stay_alone_and_large_v(on_gpu):
    M, K, N, R, L = 40, 128, 64, 16, 2
    x, y, a, b, ids, _ = adapters(M, K, N, R, L, FP, FP, 4)
    ids = torch.zeros(M, dtype=torch.int32)
    ids[10] = -1
    args = lambda xx, aa, bb: [t.to(DEV) for t in (y, xx, aa, bb, ids)]
    good = on_gpu.lora_add(*args(x, a, b))
    bad = x.clone()
    bad[3, 5], bad[10, 7], bad[20, 0] = float("nan"), float("nan"), float("inf")
    got = on_gpu.lora_add(*args(bad, a, b))
    rest = [m for m in range(M) if m not in (3, 20)]        # row 10 has no adapter: its x is not read
    assert torch.equal(got[rest], good[rest])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[20]).any()
    # v = x A^T of 1e6, beyond fp16, and B that brings it back; and v near 1e-9
    big = lora_ref(x * 30, y, a * 3000, b * 1e-4, ids, None)
    out = on_gpu.lora_add(*args((x * 30).to(FP), (a * 3000).to(FP), (b * 1e-4).to(FP)))
    big = lora_ref((x * 30).to(FP), y, (a * 3000).to(FP), (b * 1e-4).to(FP), ids, None)
    assert np.abs(big).max() < 6e4
    assert_rows_close(out, big, FP, extra=2.0 ** -15)
    small = [(x * 1e-3).to(FP), (a * 1e-2).to(FP), (b * 1e4).to(FP)]
    zero = torch.zeros_like(y)
    out = on_gpu.lora_add(*[t.to(DEV) for t in (zero, *small, ids)])
    assert_rows_close(out, lora_ref(small[0], zero, small[1], small[2], ids, None), FP, extra=2.0 ** -15)


@gpu
@pytest.mark.parametrize("M", [2, 60, 400, 700])
@pytest.mark.parametrize("R", [8, 24, 72, 128])
def test_lora_adapters_that_no_token_names_do_not_show(on_gpu, M, R):
    # slots without an adapter may hold anything, NaN too
    K, N, L = 200, 136, 5
    x, y, a, b, _, scales = adapters(M, K, N, R, L, BF, BF, 12)
    ids = torch.where(torch.arange(M) % 3 == 0, 1, 3).to(torch.int32)
    ids[M // 2] = -1
    ref = lora_ref(x, y, a, b, ids, scales)
    for i in (0, 2, 4):
        a[i], b[i], scales[i] = float("nan"), float("inf"), float("nan")
    out = on_gpu.lora_add(*[t.to(DEV) for t in (y, x, a, b, ids, scales)])
    assert_rows_close(out, ref, BF, extra=2.0 ** -15)


@gpu
@pytest.mark.parametrize("M", [64, 1500])
def test_lora_token_does_not_depend_on_its_tile(on_gpu, M):
    # the same tokens in another order and with other neighbours: the same bits
    K, N, R, L = 256, 136, 32, 3
    x, y, a, b, ids, scales = [t.to(DEV) for t in adapters(M, K, N, R, L, BF, BF, 8)]
    out = on_gpu.lora_add(y, x, a, b, ids, scales)
    p = torch.randperm(M, device=DEV)
    again = on_gpu.lora_add(y[p].contiguous(), x[p].contiguous(), a, b, ids[p].contiguous(), scales)
    assert torch.equal(again, out[p])


@gpu
@pytest.mark.parametrize("M,L", [(5, 4), (700, 4), (300, 40), (300, 1100), (5000, 500)])
def test_lora_graph_replay_streams_and_empty(on_gpu, M, L):
    K, N, R = 128, 64, 16
    x, y, a, b, ids, scales = [t.to(DEV) for t in adapters(M, K, N, R, L, BF, BF, 6)]
    ws = torch.full((on_gpu.lora_add_workspace_bytes(M, L) + 256,), 0x5A, device=DEV, dtype=torch.uint8)
    need = ws.numel() - 256
    out = torch.empty_like(y)
    side = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        on_gpu.lora_add(y, x, a, b, ids, scales, workspace=ws[:need], out=out)
    for s in range(3):
        x.copy_(torch.randn_like(x))
        ids.copy_(torch.randint(-1, L, (M,), device=DEV, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, on_gpu.lora_add(y, x, a, b, ids, scales))
    assert (ws[need:] == 0x5A).all()
    torch.cuda.synchronize()
    got = on_gpu.lora_add(y, x, a, b, ids, scales, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    assert on_gpu.lora_add(y[:0], x[:0], a, b, ids[:0], scales).shape == (0, N)


# ------------------------------------------------------------- all together

@gpu
@pytest.mark.parametrize("M", [3, 40])
def test_a_decode_step_with_adapters_and_experts(on_gpu, M):
    """A shared W4A4 projection with per-request adapters in place, then an expert layer on its output."""
    ck, K, E, k, I, R, L = on_gpu, 256, 8, 2, 128, 16, 3
    from bit_quantized_linear_rotate_b200 import workloads as WL
    d = WL.small_linear_inputs(M, K, K, seed=M)
    x, y0, a, b, ids, scales = adapters(M, K, K, R, L, BF, BF, M)
    gu, dn = experts(E, K, I, 64, BF, M)
    router = torch.randn((E, K), generator=torch.Generator().manual_seed(0)).to(BF)
    xd = d["x"].to(DEV)
    y = ck.linear_w4a4(xd, d["w_packed"].to(DEV), d["w_scale"].to(DEV), 64)
    base = y.clone()
    ck.lora_add(y, xd, a.to(DEV), b.to(DEV), ids.to(DEV), scales.to(DEV), out=y)
    logits = torch.matmul(y.float(), router.to(DEV).float().t())
    out = ck.moe_awq_w4a16(y, logits, k, *to_dev(gu), *to_dev(dn))
    assert_rows_close(y, lora_ref(d["x"], base.cpu(), a, b, ids, scales), BF, extra=2.0 ** -15)
    w, chosen = O.moe_route(f64(logits), k, True)
    assert_rows_close(out, moe_ref(y, torch.tensor(chosen), torch.tensor(w), gu, dn, 64), BF)


@gpu
def test_one_expert_agrees_with_the_awq_gemv(on_gpu):
    # the same weights as three plain projections: x Wg^T and x Wu^T by the GEMV, h rounded to bf16 there
    T, K, I = 4, 256, 128
    gu, dn = experts(1, K, I, 64, BF, 21)
    x = torch.randn((T, K), device=DEV).to(BF)
    one = torch.zeros((T, 1), device=DEV, dtype=torch.int32)
    out = on_gpu.moe_experts_awq_w4a16(x, one, torch.ones((T, 1), device=DEV), *to_dev(gu), *to_dev(dn))
    q, s, z = (t[0].to(DEV) for t in gu)
    y = on_gpu.gemv_awq_w4a16(x, q, s, z).float()
    h = (y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]).to(BF)
    ref = on_gpu.gemv_awq_w4a16(h, *(t[0].to(DEV) for t in dn))
    # gate, up and h are rounded to bf16 there (a few 2^-8 of each, averaged over I), the output in both
    assert_rows_close(out, f64(ref), BF, extra=4 * u_of(BF))


@gpu
def test_weights_beyond_32_bit_offsets(on_gpu):
    # the last of so many experts and adapters that their bytes and elements pass 2^32; the others are zeros
    E, K, I, G = 512, 4096, 4096, 256
    gu, dn = experts(1, K, I, G, BF, 31)

    def last(part, n):
        out = torch.zeros((n, *part.shape[1:]), device=DEV, dtype=part.dtype)
        out[-1] = part[0].to(DEV)
        return out

    for T in (1, 3):
        x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).to(BF)
        ids, w = torch.full((T, 1), E - 1, dtype=torch.int32), torch.ones((T, 1))
        many = [last(t, E) for t in gu + dn]
        out = on_gpu.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *many, group_size=G)
        assert_rows_close(out, moe_ref(x, torch.zeros_like(ids), w, gu, dn, G), BF)
    del many
    L, K, N, R = 700, 64, 32768, 128
    for M in (3, 600):
        x, y, a, b, _, _ = adapters(M, K, N, R, 1, BF, BF, M)
        ids = torch.full((M,), L - 1, dtype=torch.int32)
        out = on_gpu.lora_add(y.to(DEV), x.to(DEV), last(a, L), last(b, L), ids.to(DEV))
        assert_rows_close(out, lora_ref(x, y, a, b, torch.zeros_like(ids), None), BF, extra=2.0 ** -15)


@gpu
def test_calls_from_several_threads_and_streams_at_once(on_gpu):
    import threading
    E, k, K, I, R, L = 8, 2, 256, 128, 16, 3
    gu, dn = experts(E, K, I, 64, BF, 3)
    gu, dn = to_dev(gu), to_dev(dn)
    inputs, refs = [], []
    for i, M in enumerate((1, 5, 33, 64)):
        x, y, a, b, ids, scales = [t.to(DEV) for t in adapters(M, K, K, R, L, BF, BF, i)]
        logits = torch.randn((M, E), device=DEV)
        inputs.append((x, y, a, b, ids, scales, logits))
        refs.append((on_gpu.lora_add(y, x, a, b, ids, scales), on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn)))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        x, y, a, b, ids, scales, logits = inputs[i]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [(on_gpu.lora_add(y, x, a, b, ids, scales), on_gpu.moe_awq_w4a16(x, logits, k, *gu, *dn))
                   for _ in range(40)]
        stream.synchronize()
        wrong.extend(i for u, v in got if not (torch.equal(u, refs[i][0]) and torch.equal(v, refs[i][1])))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
