"""The serving suites under the bounds-checked build (see test_gpu_debug_build.py):
after every test no index check may have failed."""

import sys

import pytest

from tests.test_gpu_debug_build import run

pytestmark = pytest.mark.gpu


def test_serving_suites_under_the_checked_build():
    r = run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_serve.py",
             "tests/test_gpu_serve_block.py"], 900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


def test_edges_under_the_checked_build():
    r = run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
             "tests/test_gpu_serve_edges.py"], 900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
