"""The example that runs the serving operators together, with its own checks."""
import pytest

from examples import branching_session

pytestmark = pytest.mark.gpu


def test_branching_session(gpu):
    # outputs are averages of unit normals: below 1 in size where more than a few keys count, so two bf16 roundings
    # (weights and result, 2^-8 each of at most a few units) stay under 2^-5
    assert branching_session.main() < 2.0 ** -5
