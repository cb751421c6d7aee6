"""Helpers of the tests of the experts' products."""
import numpy as np
import torch

MARK = 0x5A                                # byte of buffers that must stay as they were


def f64(t):
    return t.detach().to("cpu").double().numpy()


def close(got, want, err, what):
    """|got - want| <= err + the rounding of got's type (half a step)."""
    eps, tiny = torch.finfo(got.dtype).eps, torch.finfo(got.dtype).smallest_normal
    if got.dtype != torch.float32:
        tiny *= eps                        # half a step below the normal numbers
    tol = err + 1.01 * ((np.abs(want) + err) * eps / 2 + tiny)
    d = np.abs(f64(got) - want)
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(d[bad] / tol[bad]):.3g} of the bound, first at "
                           f"{np.argwhere(bad)[0]}")


def rand(rng, shape, dtype, std=1.0):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).to(dtype)


def marked(shape, dtype):
    """A device buffer of a byte pattern no kernel writes by chance."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    if t.numel():
        t.view(torch.uint8).fill_(MARK)
    return t


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == MARK).all()) if t.numel() else True


def shifted(t, by=1):
    """The same values `by` elements past an aligned address."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


def spread(rng, rows, E, empty=0.25):
    """Ascending offsets of E experts that share `rows`, some without any."""
    p = rng.exponential(size=E) * (rng.random(E) >= empty)
    p = p / p.sum() if p.sum() > 0 else np.full(E, 1.0 / E)
    counts = rng.multinomial(rows, p)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
