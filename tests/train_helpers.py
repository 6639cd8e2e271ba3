"""Helpers of the tests of the operators around the matrix update."""

import numpy as np
import torch

U32 = 2.0 ** -24   # half a step of fp32, relative


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def half_step(value, dtype) -> np.ndarray:
    """Most that rounding `value` once to dtype can change it: half a relative
    step, or half the smallest subnormal."""
    info = torch.finfo(dtype)
    tiny = info.smallest_normal * info.eps
    return np.abs(value) * (info.eps / 2) + tiny / 2


def assert_within(got, want, slack, what=""):
    """|got - want| <= slack elementwise (NaN where, and only where, want is)."""
    got = f64(got) if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    off = np.abs(got - want) - slack
    off = np.where(np.isnan(want) | (got == want), -np.inf, off)
    worst = int(np.argmax(off)) if off.size else 0
    assert off.size == 0 or off.flat[worst] <= 0, (
        f"{what}: {np.sum(off > 0)} of {off.size} out of tolerance, worst at {worst}: got "
        f"{got.flat[worst]!r}, want {want.flat[worst]!r}, allowed "
        f"{np.broadcast_to(slack, want.shape).flat[worst]!r}")


def normal(seed, shape, dtype=torch.float32, scale=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype).to(device)


def strided_rows(t, extra: int, offset: int):
    """The same values as a view whose rows lie `extra` elements further apart
    and begin `offset` elements into an allocation (surroundings NaN)."""
    rows, cols = t.reshape(-1, t.shape[-1]).shape
    store = torch.full((offset + rows * (cols + extra) + 16,), float("nan"), dtype=t.dtype,
                       device=t.device)
    view = store[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    view.copy_(t.reshape(rows, cols))
    return view, store


def untouched(store, view) -> bool:
    """Whether everything of `store` around `view` still holds NaN."""
    mask = torch.ones_like(store, dtype=torch.bool)
    at = (view.data_ptr() - store.data_ptr()) // store.element_size()
    for r in range(view.shape[0]):
        mask[at + r * view.stride(0): at + r * view.stride(0) + view.shape[1]] = False
    return bool(torch.isnan(store[mask].float()).all())
