"""The expert layer and the adapters beside entries that dwarf the rest: what a weight of zero removes
must not cost the other entries any of their bits. The adapters with v = x A^T whose last bits show.

Tolerances. Where all values are integers whose sums stay below 2^24, every 32-bit operation is
exact and the output is the exact value rounded once: the tests ask for equality. The others bound each
element by the roundings that a 32-bit evaluation makes, each at most D = 2^-23 of the sum of
magnitudes that it belongs to (the tensor cores may truncate), by the place where it happens:

* gate and up: 64 products of a block and the block's sum, two roundings for each of K / 64 blocks, 8 for the
  partial sums: (64 + 2 K / 64 + 8) D of A |x|, with A = |u - 8| s + |z|;
* h = silu(gate) up: |silu'| <= 1.1, and 4 D of |h| for the exponential, the quotient and the products;
* h enters the second product as two fp16 numbers after a power of two that brings the block's largest
  magnitude to at least 2^13: off by D of itself and by 2^-25 (half of fp16's smallest step)
  of that scale, 2^-38 of the block's largest;
* the second product: 128 products of a block and the block's sum, two roundings for each of I / 64 blocks, and
  24 for the weight, the partial sums and the slots: (128 + 2 I / 64 + 24) D of A |h| w;
* the output: half a step of its type, torch.finfo(t).eps / 2.
"""

import numpy as np
import pytest
import torch

import oracle as O

DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16
D = 2.0 ** -23
gpu = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


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


# ------------------------------------------------------------ the expert layer

def packed(u):
    """(..., n) values 0 .. 15 -> (..., n / 2) bytes, the even column in the low nibble."""
    return (u[..., 0::2] | u[..., 1::2] << 4).to(torch.uint8)


def run_experts(ck, x, ids, w, gate_up, down, G):
    parts = [t.to(DEV) for t in gate_up + down]
    return ck.moe_experts_awq_w4a16(x.to(DEV), ids.to(DEV), w.to(DEV), *parts, group_size=G)


def reference(x, ids, w, gate_up, down, G):
    num = [[m[0].numpy(), f64(m[1]), f64(m[2])] for m in (gate_up, down)]
    return O.moe_awq_w4a16(f64(x), ids.numpy(), f64(w), *num, G)


def bounded_reference(x, ids, w, gate_up, down, G):
    """The oracle's output, how far a 32-bit evaluation may be from it before the output's rounding, and the
    magnitudes that the output is a sum of."""
    ref = reference(x, ids, w, gate_up, down, G)

    def parts(m, e):
        q = np.stack((m[0][e].numpy() & 15, m[0][e].numpy() >> 4), axis=-1).reshape(m[0].shape[1], -1) - 8.0
        s, z = (np.repeat(f64(v[e]), G, axis=0).T for v in m[1:])
        return q * s + z, np.abs(q) * s + np.abs(z)

    slack, most = np.zeros_like(ref), np.zeros_like(ref)
    x, w = f64(x), f64(w)
    for e in range(gate_up[0].shape[0]):
        (W, A), (Wd, Ad) = parts(gate_up, e), parts(down, e)
        I = Wd.shape[1]
        for t, j in zip(*np.nonzero(ids.numpy() == e)):
            v, ev = W @ x[t], (64 + 2 * (W.shape[1] // 64) + 8) * D * (A @ np.abs(x[t]))
            gate, up, eg, eu = v[:I], v[I:], ev[:I], ev[I:]
            sg = O.silu(gate)
            h = sg * up
            most[t] += abs(w[t, j]) * (Ad @ np.abs(h))
            top = np.repeat(np.abs(h).reshape(-1, 64).max(axis=1), 64)
            eh = 1.1 * eg * np.abs(up) + (np.abs(sg) + 1.1 * eg) * eu + 5 * D * np.abs(h) + 2.0 ** -38 * top
            slack[t] += abs(w[t, j]) * (Ad @ eh + (128 + 2 * (I // 64) + 24) * D * (Ad @ (np.abs(h) + eh)))
    return ref, slack, most


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K,I,G", [(192, 128, 64), (384, 320, 64), (256, 384, 128), (512, 256, 256)])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 20, 64])
@pytest.mark.parametrize("outlier", [1, 1024, 16384])
def test_moe_integers_come_through_exactly(on_gpu, T, K, I, G, dtype, outlier):
    # x of 48 ones and one large entry that no row but one has a weight for; that row makes one large entry of
    # h, which no output has a weight for
    E, cx, ch = 2, 75, 37
    g = torch.Generator().manual_seed(T * 1000 + K)
    x = torch.zeros((T, K))
    for t in range(T):
        x[t, torch.randperm(K, generator=g)[:48]] = 1
    x[:, cx] = outlier
    u = torch.randint(0, 16, (E, 2 * I, K), generator=g)
    u[:, :I] = 9                                            # gate = sum(x) >= 47: silu(gate) = gate in 32 bits
    u[:, :, cx] = 8
    u[:, ch, cx] = u[:, I + ch, cx] = 9
    z = torch.randint(-1, 2, (E, K // G, 2 * I), generator=g).double()
    z[:, :, :I] = 0
    z[:, cx // G] = 0
    gate_up = (packed(u), torch.ones(z.shape).to(dtype), z.to(dtype))
    u = torch.randint(0, 16, (E, K, I), generator=g)
    u[:, :, ch] = 8
    z = torch.randint(-1, 2, (E, I // G, K), generator=g).double()
    z[:, ch // G] = 0
    down = (packed(u), torch.full(z.shape, 2.0 ** -7).to(dtype), (z * 2.0 ** -7).to(dtype))
    x = x.to(dtype)
    ids = torch.tensor([[1, 0], [0, -1], [-1, 1]], dtype=torch.int32)[torch.arange(T) % 3]
    w = torch.tensor([[1.0, -1.0], [1.0, 1.0], [1.0, -1.0]])[torch.arange(T) % 3].contiguous()
    ref, _, most = bounded_reference(x, ids, w, gate_up, down, G)
    assert (ref * 128 == np.round(ref * 128)).all() and most.max() * 128 < 2 ** 23 and np.abs(ref).max() < 6e4
    out = run_experts(on_gpu, x, ids, w, gate_up, down, G)
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(dtype))


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,K,I,G", [(1, 512, 256, 64), (2, 256, 320, 64), (5, 256, 256, 256), (12, 384, 192, 64),
                                     (40, 256, 256, 128)])
@pytest.mark.parametrize("spread", ["even", "channels", "spikes"])
def test_moe_each_element(on_gpu, T, K, I, G, dtype, spread):
    # "channels": a few columns of x are thousands of times as large as the others and most rows have no weight for
    # them; "spikes": the same of h
    E = 4
    g = torch.Generator().manual_seed(T + K)

    def part(rows, cols):
        return (torch.randint(0, 16, (E, rows, cols), generator=g),
                (torch.rand((E, cols // G, rows), generator=g) * 0.009 + 0.001).to(dtype),
                (torch.randn((E, cols // G, rows), generator=g) * 0.01).to(dtype))

    gate_up, down = part(2 * I, K), part(K, I)
    x = torch.randn((T, K), generator=g)
    if spread == "channels":
        for c, v in ((3, 3000.0), (70, -12345.0), (K - 1, 600.0)):
            x[:, c] = v
            gate_up[0][:, 1:, c] = 8
            gate_up[2][:, c // G, 1:] = 0
    if spread == "spikes":
        x = x.abs()
        for c in (2, 129, I - 1):
            gate_up[0][:, c], gate_up[0][:, I + c] = 12, 13
            gate_up[1][:, :, c] = gate_up[1][:, :, I + c] = 1.0
            down[0][:, :, c] = 8
            down[2][:, c // G] = 0
        x = x / 4
    x = x.to(dtype)
    gate_up, down = (packed(gate_up[0]), *gate_up[1:]), (packed(down[0]), *down[1:])
    ids = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(T)]).to(torch.int32)
    w = torch.rand((T, 2), generator=g) + 0.1
    ref, slack, _ = bounded_reference(x, ids, w, gate_up, down, G)
    out = f64(run_experts(on_gpu, x, ids, w, gate_up, down, G))
    u = torch.finfo(dtype).eps / 2
    bound = slack + u * (np.abs(ref) + slack) + torch.finfo(dtype).tiny
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= bound).all(), f"{(np.abs(out - ref) / bound).max():.3g} of the bound"


# ---------------------------------------------------------------- the adapters

LORA = [(1, 3), (40, 3), (600, 3), (1500, 2), (300, 1100)]    # few tokens, tiles of 16 and of 128, listed tiles


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,L", LORA)
@pytest.mark.parametrize("R", [8, 64, 72, 128])
def test_lora_integers_come_through_exactly(on_gpu, M, L, R, dtype):
    # v of up to 20 bits, whose last bits show in the sums
    K, N = 64, 136
    g = torch.Generator().manual_seed(M + R)
    x = torch.randint(-127, 128, (M, K), generator=g).to(dtype)
    y = torch.randint(-127, 128, (M, N), generator=g).to(dtype)
    a = torch.randint(-127, 128, (L, R, K), generator=g).to(dtype)
    b = torch.randint(-1, 2, (L, N, R), generator=g).to(dtype)
    ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32).sort().values
    scales = torch.full((L,), 2.0 ** -8)
    ref = O.lora_add(f64(y), f64(x), f64(a), f64(b), ids.numpy(), f64(scales))
    assert np.abs(ref).max() < 2 ** 15                      # and so below 2^23 in steps of 2^-8
    out = on_gpu.lora_add(*[t.to(DEV) for t in (y, x, a, b, ids, scales)])
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(dtype))


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,L", LORA)
@pytest.mark.parametrize("R", [8, 72])
def test_lora_ranks_that_cancel(on_gpu, M, L, R, dtype):
    # v = (1 + 2^-10 + 2^-20, -1 - 2^-10, 0 ...): what is left of their sum is 2^-20
    K, N = 40, 72
    x, y = torch.zeros((M, K), dtype=dtype), torch.zeros((M, N), dtype=dtype)
    a, b = torch.zeros((L, R, K), dtype=dtype), torch.ones((L, N, R), dtype=dtype)
    x[:, :3] = 1.0
    a[:, 0, :3] = torch.tensor([1.0, 2.0 ** -10, 2.0 ** -20])
    a[:, 1, :3] = torch.tensor([-1.0, -(2.0 ** -10), 0.0])
    ids = torch.arange(M, dtype=torch.int32) * L // M
    out = on_gpu.lora_add(*[t.to(DEV) for t in (y, x, a, b, ids)])
    assert (out == 2.0 ** -20).all()


@gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,L", LORA)
@pytest.mark.parametrize("R", [8, 40, 72, 128])
def test_lora_infinity_that_the_formula_keeps(on_gpu, M, L, R, dtype):
    # x with an infinity, all weights positive: v and the output are that infinity, whatever the rank
    K, N = 72, 40
    x, y = torch.ones((M, K), dtype=dtype), torch.ones((M, N), dtype=dtype)
    a, b = torch.full((L, R, K), 0.5, dtype=dtype), torch.full((L, N, R), 0.25, dtype=dtype)
    x[0, 5] = float("inf")
    x[M // 2, 70] = -float("inf")
    ids = torch.arange(M, dtype=torch.int32) * L // M
    out = on_gpu.lora_add(*[t.to(DEV) for t in (y, x, a, b, ids)]).cpu()
    ref = torch.full((M, N), 1 + R * K * 0.125, dtype=torch.float64)
    ref[0] = float("inf")
    ref[M // 2] = -float("inf")
    if M == 1:
        ref[0] = float("nan")                               # both infinities in one row
    torch.testing.assert_close(out.double(), ref.to(dtype).double(), rtol=0, atol=0, equal_nan=True)


# ------------------------------------------------------------- several callers

@gpu
def test_every_call_of_every_thread_returns_its_result(on_gpu):
    # a call that raises in its thread fails the test, and so does one that is missing
    from concurrent.futures import ThreadPoolExecutor
    E, k, K, I, R, L, rounds = 8, 2, 256, 128, 16, 3, 40
    g = torch.Generator().manual_seed(3)

    def part(rows, cols):
        return [torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8).to(DEV),
                (torch.rand((E, cols // 64, rows), generator=g) * 0.009 + 0.001).to(BF).to(DEV),
                (torch.randn((E, cols // 64, rows), generator=g) * 0.01).to(BF).to(DEV)]

    experts = part(2 * I, K) + part(K, I)
    a, b = ((torch.randn(s, generator=g) / 16).to(BF).to(DEV) for s in ((L, R, K), (L, K, R)))
    inputs = []
    for M in (1, 5, 33, 64):
        x, y = (torch.randn((M, K), generator=g).to(BF).to(DEV) for _ in range(2))
        ids = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32).to(DEV)
        inputs.append((x, y, ids, torch.randn((M, E), generator=g).to(DEV)))

    def calls(x, y, ids, logits):
        return (on_gpu.lora_add(y, x, a, b, ids), on_gpu.moe_awq_w4a16(x, logits, k, *experts),
                *on_gpu.moe_route(logits, k))

    refs = [calls(*v) for v in inputs]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [calls(*inputs[i]) for _ in range(rounds)]
        stream.synchronize()
        return sum(all(torch.equal(p, q) for p, q in zip(one, refs[i])) for one in got)

    with ThreadPoolExecutor(len(inputs)) as pool:
        futures = [pool.submit(work, i) for i in range(len(inputs))]
        assert [f.result() for f in futures] == [rounds] * len(inputs)
