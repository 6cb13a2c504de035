"""The 8-bit append on both sides of the borders between its forms (CTAs of 16 warps for large
calls whose runs of 16 tokens are few or wide, of eight otherwise), byte for byte."""
import pytest

from test_fp8_gpu import append_case, env, run_append  # noqa: F401  (env: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held,new,Hq,Hkv,d", [
    ([5, 0], [1000, 900], 64, 8, 64),        # few runs of 160 KB
    ([7] * 4, [1900] * 4, 80, 8, 64),        # many of 192 KB
    ([7] * 4, [1900] * 4, 78, 8, 64),        # ... and a little less
    ([7] * 4, [1900] * 4, 32, 8, 128),       # many of 192 KB
    ([7] * 4, [1900] * 4, 30, 8, 128),
    ([0, 3], [1500, 1400], 32, 8, 128)])     # between: more runs than SMs
def test_append_forms(env, held, new, Hq, Hkv, d):
    run_append(env, append_case(950, held, new, Hq, Hkv, d), Hkv, d, (d // 2,))
