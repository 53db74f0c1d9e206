"""A context is made, asked for its sizes and closed without torch; only the calls that take tensors need it."""
import subprocess
import sys

import pytest

from conftest import ROOT

from kv_cache_quantization_tq_gb300.build import build

build()

BODY = """
import sys
sys.modules["torch"] = None  # an import of it fails
sys.path.insert(0, {root!r})
import kv_cache_quantization_tq_gb300 as tq
from kv_cache_quantization_tq_gb300 import binding
{fake}
for layout, size in ((tq.TQ_LAYOUT_MAIN, 16 * 52), (tq.TQ_LAYOUT_ALT, 16 * 98), (tq.TQ_LAYOUT_DENSE, 64 * 64)):
    ctx = tq.Context(layout, 64, 4, 2)
    assert ctx.cfg.layout == layout and ctx.page_bytes == size, (layout, ctx.page_bytes)
    ctx.close()
"""

FAKE = """
class Library:  # the calls that need a GPU
    def __getattr__(self, name):
        return getattr(real, name)
    def tq_create(self, cfg, out):
        self.cfg = cfg._obj
        return 0
    def tq_page_bytes(self, ptr):
        return 16 * binding.tq_config_check(self.cfg)
    def tq_ctx_device(self, ptr):
        return 0
real, binding.lib = binding.lib, Library()
"""


def run(fake):
    r = subprocess.run([sys.executable, "-c", BODY.format(root=ROOT, fake=fake)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_with_a_library_that_needs_no_gpu():
    run(FAKE)


@pytest.mark.gpu
def test_with_the_library():
    run("")


def test_the_device_of_no_context():
    from kv_cache_quantization_tq_gb300 import binding

    assert binding.lib.tq_ctx_device(None) == -1
