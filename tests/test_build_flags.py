"""Which sources are compiled with NaN handling (CPU)."""
import os

from confidence_block_unmasking_amd import build


def test_calls_that_promise_nan_are_built_with_it():
    """dllm_logprobs writes NaN for slots without a distribution, as a difference of infinities or a sum
    with NaN in it; a compiler told that there is no NaN may make anything of either."""
    seen = {os.path.basename(s) for s in build.SOURCES}
    assert set(build.NONFINITE_SOURCES) <= seen
    for s in build.SOURCES:
        nans = not any("honor-nans" in f or "finite-math" in f or f in ("-ffast-math", "-Ofast") for f in build.flags(s))
        assert nans == (os.path.basename(s) in ("logprobs.hip", "embed.hip")), s
        assert "-packed-fp32-ops" in build.flags(s)
