"""References in 64 bits for the training operators' tests, and the bounds
that their results are held to."""

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of a rounding


def offsets_of(counts, device="cuda"):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts).cumsum(0)
    return off.to(device)


def sum_bound(mag, n, ref, out_dtype):
    """|error| of a sum of n exact products, magnitudes adding up to `mag`:
    every fp32 addition is off by at most a whole step of the running sum
    (2^-23: the matrix unit may cut instead of rounding), and the result is
    rounded once to out_dtype."""
    return (n + 2) * 2.0 ** -23 * mag + U[out_dtype] * ref.abs() * 1.01


def gmm_ref(form, counts, lhs, rhs):
    """(value, sum of magnitudes, longest sum) in 64 bits."""
    lo, val, mag, longest = 0, [], [], 1
    for e, c in enumerate(counts):
        x = lhs[lo:lo + c].double()
        if form == "dw":
            y = rhs[lo:lo + c].double()
            val.append(x.t() @ y)
            mag.append(x.abs().t() @ y.abs())
            longest = max(longest, c)
        else:
            w = rhs[e].double()
            w = w.t() if form == "fwd" else w
            val.append(x @ w)
            mag.append(x.abs() @ w.abs())
            longest = max(longest, w.shape[0])
        lo += c
    join = torch.stack if form == "dw" else torch.cat
    return join(val), join(mag), longest
