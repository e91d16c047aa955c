"""Grouped operators on tensors whose offsets pass 32 bits, against fp64 on the rows that sit past them.

Tolerances as in test_gpu_grouped.py and test_gpu_lora.py; inputs are made on the device.
"""
import numpy as np
import pytest
import torch

from tests.qlhelpers import dev

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def _near(got, ref, bound, dtype):
    err = (got.double() - ref).abs()
    bound = bound + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * (ref.abs() + bound) + 1e-37
    assert bool((err <= bound).all()), float((err / bound).max())


def _codes(G, N, K, gen):
    """Codes of all groups, random bytes, filled in pieces (int32 words)."""
    c = torch.empty(G, N, 3 * K // 4, dtype=torch.uint8, device="cuda")
    c.view(-1).view(torch.int32).random_(-2 ** 31, 2 ** 31 - 1, generator=gen)
    return c


def _weights(codes, lut, g, K):
    """W_g fp64 [N, K] from 4 six-bit codes per 3 bytes, little endian."""
    b = codes[g].view(codes.shape[1], K // 4, 3).to(torch.int64)
    v = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16
    idx = torch.stack([v >> 6 * e & 63 for e in range(4)], -1).view(codes.shape[1], K)
    return torch.gather(lut[g].double(), 1, idx)


@pytest.mark.parametrize("K", [5120, 1348])                  # tensor cores, plain cores
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_and_outputs_past_32_bits(ql, K, dtype):
    gen = torch.Generator("cuda").manual_seed(K)
    G, N = (512, 2320) if K == 5120 else (1024, 4400)
    codes = _codes(G, N, K, gen)
    assert codes.numel() > 2 ** 32
    lut = torch.randn(G, N, 64, generator=gen, device="cuda").bfloat16()
    x = torch.randn(9, K, generator=gen, device="cuda").bfloat16()
    Y = 2 ** 32 // (N * dtype.itemsize) + 20
    y = torch.full((Y, N), 3.0, dtype=dtype, device="cuda")
    counts = np.zeros(G, dtype=np.int64)
    counts[[0, G - 2, G - 1]] = 2, 3, 4
    offsets = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    rows = torch.tensor([0, Y - 1, 5, Y - 3, Y - 2, 7, Y - 8, Y - 9, 1], **I32)
    ql.benq_grouped_linear(codes, lut, x, offsets, y, y_rows=rows)
    ql.ql_check()
    for g, sl in ((0, slice(0, 2)), (G - 2, slice(2, 5)), (G - 1, slice(5, 9))):
        W = _weights(codes, lut, g, K)
        xs = x[sl].double()
        _near(y[rows[sl].long()], xs @ W.T, (K / 16 + 32) * 2.0 ** -22 * (xs.abs() @ W.abs().T), dtype)
    y[rows.long()] = 3.0
    assert bool((y == 3.0).all())


def test_combine_past_32_bits(ql):
    T, k, N = 54000, 8, 5120
    gen = torch.Generator("cuda").manual_seed(1)
    y = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert y.numel() * 2 > 2 ** 32
    experts = torch.randint(-1, 4, (T, k), generator=gen, **I32)
    w = torch.rand(T, k, generator=gen, device="cuda")
    out = torch.empty(T, N, device="cuda")
    ql.moe_combine(y, experts, w, out)
    ql.ql_check()
    for t in (0, T // 2, 52430, T - 2, T - 1):
        on = (experts[t] >= 0).double() * w[t].double()
        rows = y[t * k:(t + 1) * k].double()
        _near(out[t], on @ rows, (k + 2) * 2.0 ** -24 * (on @ rows.abs()), torch.float32)


@pytest.mark.parametrize("T,G,N,r,K,dtype", [
    (6, 1024, 4100, 256, 17408, torch.bfloat16),             # A above 4 GB
    (3200, 64, 262176, 128, 256, torch.bfloat16),            # B above 4 GB, tensor copies
    (2_200_000, 2, 1024, 8, 16, torch.bfloat16),             # y above 4 GB
    (2_200_000, 2, 520, 4, 16, torch.float32),               # the same, more tiles than a grid's second dimension holds
])
def test_lora_past_32_bits(ql, T, G, N, r, K, dtype):
    gen = torch.Generator("cuda").manual_seed(T + r)
    A = (torch.empty(G, r, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)) * K ** -0.5
    B = torch.empty(G, N, r, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    y = torch.empty(T, N, dtype=dtype, device="cuda").normal_(generator=gen)
    assert max(A.numel() * 2, B.numel() * 2, y.numel() * dtype.itemsize) > 2 ** 32
    index = torch.randint(0, G, (T,), generator=gen, **I32)
    index[:4] = G - 1
    order, offsets = torch.empty(T, **I32), torch.empty(G + 1, **I32)
    room = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda") if n else None  # noqa: E731
    ql.group_rows(index, G, order, offsets, workspace=room(ql.group_rows_workspace_bytes(T, G)))
    pick = torch.cat([torch.arange(4), torch.arange(T - 2, T)]).cuda()
    y0 = y[pick].double()
    ql.lora_add([(A, B, y)], x, order, offsets, workspace=room(ql.lora_workspace_bytes(1, T, r)))
    ql.ql_check()
    for i, t in enumerate(pick.tolist()):
        a, b, v = A[index[t]].double(), B[index[t]].double(), x[t].double()
        ref, s = y0[i] + b @ (a @ v), b.abs() @ (a.abs() @ v.abs())
        _near(y[t], ref, ((K / 8 + 64 + r + 8) * 2.0 ** -23 + (2.0 ** -17 if dtype == torch.bfloat16 else 2.0 ** -25)) * s, dtype)
