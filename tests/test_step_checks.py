"""The row checks of the serving step's GPU tests see what is planted in them (no GPU)."""
import numpy as np
import pytest

pytest.importorskip("kv_cache_quantization_turbo_gb300.tq", reason="libtq.so not built")
import step_checks as K  # noqa: E402


def rows():
    want = np.random.default_rng(0).standard_normal((6, 2, 64))
    want[4] = 0.0
    return want.copy(), want, np.full((6, 2), 1e-3)


def nan_row(x):
    x[3, 1] = np.nan


def one_nan(x):
    x[3, 1, 5] = np.nan


def infinite(x):
    x[0, 0, 0] = np.inf


def far_off_beside_nan(x):
    x[2] *= 2.0
    x[3, 1] = np.nan


def far_off(x):
    x[5, 0] *= 1.002


def not_empty(x):
    x[4, 1, 63] = 1e-30


def test_rows_within_the_bound_pass():
    got, want, bound = rows()
    K.assert_rows(got * (1 + 5e-4), want, bound)


@pytest.mark.parametrize("plant", [nan_row, one_nan, infinite, far_off_beside_nan, far_off, not_empty])
def test_planted_mistakes_are_seen(plant):
    got, want, bound = rows()
    plant(got)
    with pytest.raises(AssertionError):
        K.assert_rows(got, want, bound)
