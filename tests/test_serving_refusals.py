"""Arguments of the serving calls at the edge of what they accept, without a GPU."""

from test_serving_checks import attn, lib  # noqa: F401


def test_a_scale_that_passes_f32_in_log2_units_is_refused(lib):  # noqa: F811
    # p = 2^(scale log2(e) q.k): 2.4e38 log2(e) is infinite in f32, and infinity times a zero score a NaN
    for scale in (2.4e38, 3.4e38):
        assert attn(lib, scale=scale) == -1
