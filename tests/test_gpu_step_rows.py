"""The attention tests of test_gpu_step.py once more, with every output row checked for itself.

check_attend() there keeps the largest excess over the bound with Python's max(), which passes over NaN, and takes a
sequence's largest with NumPy's, which a single NaN hides: a row of NaN, or any row beside one, went unseen.  Here the
same calls go through step_checks.check_attend().
"""
import pytest

import step_checks as K
import test_gpu_step as T
from test_gpu_step import (ctxs, test_attend_contiguous_cache_and_layers,  # noqa: F401  (collected here too)
                           test_attend_documents_and_empty_rows, test_attend_few_rows,
                           test_attend_few_rows_contiguous_and_layers,
                           test_attend_few_rows_documents_types_and_outliers,
                           test_attend_few_rows_score_modifications, test_attend_few_rows_turbo_values,
                           test_attend_formats_and_dims, test_attend_full_width_sampled_rows,
                           test_attend_prefixes_outside_the_sequence_and_rising_bias, test_attend_scale_of_any_sign,
                           test_attend_score_modifications, test_attend_shapes, test_attend_types)


pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def every_row(monkeypatch):
    monkeypatch.setattr(T, "check_attend", K.check_attend)

