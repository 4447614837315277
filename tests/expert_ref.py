"""Plain implementations of the expert-side operators in 64 bits, with the error
bounds of a float32 computation beside them.  No library code is used.

Bounds.  A rounding to type t is off by at most half a step,
torch.finfo(t).eps / 2 relative to the value: U = 2^-24 for float32, 2^-8 for
bf16, 2^-4 for e4m3 (plus half the subnormal step, 2^-10, near zero).  A sum of
float32 terms along a chain of n additions is off by at most about n U times
the sum of the terms' magnitudes; sums inside the bf16 matrix instruction are
taken at twice that, since its inner additions may truncate instead of rounding.

The 8-bit matrix instruction lines each 8 adjacent products up with the largest
of them and drops what lies 2^-13 of it and further below.  Each of the 8 loses
at most 2^-13 of the group's largest, and the largest of all groups together
are at most the sum of all magnitudes M: it is off by at most 8 * 2^-13 M.  On
random values the losses mostly cancel; RMS_BF16 is what is left then.
"""

import torch

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
U32 = 2.0 ** -24
UBF16 = torch.finfo(torch.bfloat16).eps / 2
UE4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2
U8 = 8 * 2.0 ** -13
# The error of a rounding to bf16 is spread evenly over half a step on both sides: at most 2^-8 / sqrt(3) of the value
# in the square mean (for values just above a power of two; 2^-8 / sqrt(7) when they are spread evenly up to the next).
RMS_BF16 = UBF16 / 3 ** 0.5
E4M3_SUB = 2.0 ** -10  # half of the smallest e4m3 step


def blocks(n):
    return -(-n // BLOCK)


def routing(T, E, k, seed, drop=0.0, device="cpu"):
    """k distinct experts per token; dropped entries hold -1."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids.to(device)


def layout(ids, E):
    """offsets [E + 1] and dest_row [T, k] of the stable order by expert."""
    flat = ids.reshape(-1).long().cpu()
    dest = torch.full((flat.numel(),), -1, dtype=torch.int32)
    offsets, at = [0], 0
    for e in range(E):
        here = torch.nonzero(flat == e).reshape(-1)
        dest[here] = torch.arange(at, at + here.numel(), dtype=torch.int32)
        at += here.numel()
        offsets.append(at)
    return torch.tensor(offsets, dtype=torch.int32).to(ids.device), dest.view(ids.shape).to(ids.device)


def quantise(v):
    """The rule of the library in float32, step by step: q = e4m3(v * (448 /
    amax)), scale = amax / 448 per block."""
    v = v.float()
    q = torch.empty(v.shape, dtype=torch.float8_e4m3fn, device=v.device)
    scale = torch.empty(v.shape[0], blocks(v.shape[1]), device=v.device)
    for b in range(blocks(v.shape[1])):
        part = v[:, b * BLOCK : (b + 1) * BLOCK]
        mag = torch.where(torch.isnan(part), 0.0, part.abs())
        amax = mag.amax(1).clamp_min(AMAX_FLOOR)
        # (tensor by tensor: a division by a Python number would multiply by its rounded inverse on a GPU)
        most = torch.full_like(amax, E4M3_MAX)
        q[:, b * BLOCK : (b + 1) * BLOCK] = (part * (most / amax)[:, None]).to(torch.float8_e4m3fn)
        scale[:, b] = amax / most
    return q, scale


def random_rows(rows, n, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(rows, n, generator=g, device=device) * torch.exp(torch.randn(rows, 1, generator=g, device=device))
    return quantise(x)


def random_weights(E, N, K, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)
    q = (torch.randn(E, N, K, generator=g, device=device) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    s = torch.exp(torch.randn(E, blocks(N), blocks(K), generator=g, device=device)) / (100.0 * K ** 0.5)
    return q, s


def product(a, a_scale, offsets, b, b_scale, eight_bit=False):
    """(p, bound): the experts' products in 64 bits, NaN in rows that no expert
    holds, and how far a float32 computation by blocks may be from them, its
    inner sums from the bf16 or the 8-bit matrix instruction."""
    p, mag = terms(a, a_scale, offsets, b, b_scale)
    # inner sums of 128, the two scale roundings and their product, the sum over the blocks
    inner = U8 if eight_bit else 2 * BLOCK * U32
    return p, mag * (inner + (blocks(a.shape[1]) + 3) * U32)


def terms(a, a_scale, offsets, b, b_scale):
    """(p, mag): the products, and the sum of the magnitudes of each one's
    terms (0 in rows that no expert holds)."""
    rows, K = a.shape
    E, N, _ = b.shape
    p = torch.full((rows, N), float("nan"), dtype=torch.float64, device=a.device)
    mag = torch.zeros((rows, N), dtype=torch.float64, device=a.device)
    off = offsets.tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        ae, we = a[lo:hi].double(), b[e].double()
        ae = ae * a_scale[lo:hi].double().repeat_interleave(BLOCK, 1)[:, :K]
        we = we * b_scale[e].double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
        p[lo:hi] = ae @ we.t()
        mag[lo:hi] = ae.abs() @ we.abs().t()
    return p, mag


def magnitude(a, a_scale, offsets, b, b_scale):
    return terms(a, a_scale, offsets, b, b_scale)[1]


def swiglu(p, bound):
    """(h, bound) of SiLU(gate) * up; |d SiLU| <= 1.1."""
    gate, up = p.chunk(2, dim=1)
    bg, bu = bound.chunk(2, dim=1)
    silu = gate * torch.sigmoid(gate)
    h = silu * up
    # exp, the addition, the quotient and the product: a few roundings, exp's argument among them
    return h, 1.1 * bg * (up.abs() + bu) + silu.abs() * bu + (8 + gate.abs()) * U32 * h.abs()


def _valid(dest, rows):
    t, j = torch.nonzero((dest >= 0) & (dest < rows), as_tuple=True)
    return t, j, dest[t, j].long()


def dispatch(x, dest, rows):
    out = torch.zeros(rows, x.shape[1], dtype=torch.float64, device=x.device)
    t, _, r = _valid(dest, rows)
    out[r] = x.double()[t]
    return out


def combine(y, dest, w):
    out = torch.zeros(dest.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    t, j, r = _valid(dest, y.shape[0])
    return out.index_add_(0, t, w.double()[t, j][:, None] * y.double()[r])


def combine_backward(dout, y, dest, w):
    dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    dw = torch.zeros(dest.shape, dtype=torch.float64, device=y.device)
    t, j, r = _valid(dest, y.shape[0])
    dy[r] = w.double()[t, j][:, None] * dout.double()[t]
    dw[t, j] = (dout.double()[t] * y.double()[r]).sum(1)
    return dy, dw


def dispatch_backward(drecv, dest):
    dx = torch.zeros(dest.shape[0], drecv.shape[1], dtype=torch.float64, device=drecv.device)
    t, _, r = _valid(dest, drecv.shape[0])
    return dx.index_add_(0, t, drecv.double()[r])
