"""The example of a layer over the paged cache: what it captures, and in a process of its own."""
import os
import subprocess
import sys

import pytest

from bit_weight_only_mxfp4_gb300 import thinmx

from . import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gu.ensure_lib()
    assert gu.device_error() == 0


def test_example_captures_only_calls_that_were_made(monkeypatch):
    """A call may be captured once it has been made on the device: the example keeps to it, for every entry point and
    number of rows."""
    import torch
    from examples import paged_layer
    made, early = set(), []

    def watch(name, rows):
        call = getattr(thinmx, name)

        def watched(*a, **k):
            key = (name, a[rows] if rows is not None else None)
            if not torch.cuda.is_current_stream_capturing():
                made.add(key)
            elif key not in made:
                early.append(key)
            return call(*a, **k)
        monkeypatch.setattr(thinmx, name, watched)

    for name, rows in (("tt_bf16_matvec", 4), ("tt_mxfp4_swiglu_matvec", 4), ("tt_paged_rope_append", None),
                       ("tt_paged_decode_attention", None), ("tt_paged_prefill_attention", None)):
        watch(name, rows)
    paged_layer.serve(False, steps=3)
    assert made and not early, early


@pytest.mark.parametrize("fp8", [False, True])
def test_example_in_a_process_of_its_own(fp8):
    """Nothing has been called on the device before the example: what it captures, it has called once."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "paged_layer.py"), "--steps", "5"] +
                       (["--fp8"] if fp8 else []), capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
    assert float(r.stdout.split()[-1]) <= 7 * 2.0 ** -8
