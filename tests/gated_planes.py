"""fp32 products of the gated projections as the tensor cores form them, and the bound that tells
each of their parts from its absence.

The kernels take an fp32 number x as bf16 planes x0 + x1 + x2 and sum six products of planes, in
runs of four stages of 64 steps of the contraction.  Inputs of `planed` are positive with all
planes positive: x0 in [1, 1.25), x1 in [1.5, 1.98] 2^-9 and x2 in [1.5, 1.97] 2^-18, so that
nothing cancels, whatever the sum's length: a missing product of planes takes 2^-18 of the result
or more (over 64 steps of 2^-24), in half of the contraction half of that.

Bound, in units of 2^-24 of the (positive) result:
  17    a run's x0 y0, the last product, in 16 steps of 16 terms: each cuts the sum off by less
        than 2^-23 of what it is then, on average 8.5 / 16 of the run's
   1    the other products before it, whose sums are below 2^-7 of the run's: 80 steps
   2    x1 y2, x2 y1 and x2 y2, which are left out: below 4 * 2^-27 twice, and 4 * 2^-36
   1    rounding to nearest at the store
   7    terms that a step aligns before it adds them (a few bits below the sum's last)
   1/2  for every sum of runs or parts, to nearest, of a sum that has half its size on average
"""
import torch


def bound(sums):
    return (28 + sums / 2) * 2.0 ** -24


def planed(*shape, seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    draw = lambda lo, hi, step: torch.randint(lo, hi, shape, generator=g).double() * step
    x = (draw(128, 160, 2.0 ** -7) + draw(192, 254, 2.0 ** -16) + draw(48, 64, 2.0 ** -23))
    assert torch.equal(x.float().double(), x)
    return x.float()


def planes(x):
    """The three bf16 numbers of each element, in 64 bits."""
    out, left = [], x.double()
    for _ in range(3):
        out.append(left.bfloat16().double())
        left = left - out[-1]
    return out


PRODUCTS = [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]   # small ones first
STEP, STAGE, RUN = 16, 64, 4


def _cut(x):
    """Positive numbers cut off after 24 bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.floor(m * 2.0 ** 24), e - 24)


def emulated(operands, leave_out=lambda operand, run, product: False, run_stages=RUN):
    """Sum over the operands of A B^T, A (M, K) and B (N, K) fp32, as the kernels form it."""
    total = None
    for o, (A, B) in enumerate(operands):
        a, b, K = planes(A), planes(B), A.shape[1]
        for u, k0 in enumerate(range(0, K, run_stages * STAGE)):
            acc = torch.zeros((A.shape[0], B.shape[0]), dtype=torch.float64)
            for i, j in PRODUCTS:
                if leave_out(o, u, (i, j)):
                    continue
                for k in range(k0, min(k0 + run_stages * STAGE, K), STEP):
                    acc = _cut(acc + a[i][:, k:k + STEP] @ b[j][:, k:k + STEP].T)
            total = acc.float() if total is None else total + acc.float()
    return total


def exact(operands):
    return sum(A.double() @ B.double().T for A, B in operands)


def off(got, want):
    """Largest error relative to the result."""
    return float(((got.double().cpu() - want) / want).abs().max())
