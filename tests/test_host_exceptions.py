"""Host memory that runs out inside a C entry point comes back as FA_ERR_ALLOC, and
does not end the process: the planning calls in a child process whose address space
leaves no room for the work list (68 GB)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import resource
import masked_attention_fa_b200 as fa
fa.load_library()
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
d = fa.make_desc("BNSD", 65000, 65535, 1, 1, 64, 2)
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 29), used + (1 << 29)))
try:
    fa.{call}(d)
except fa.FaError as e:
    print(e.name)
d = fa.make_desc("BNSD", 1, 2, 128, 128, 64, 2)
print(fa.fa_visible_pairs(d))
"""


@pytest.mark.parametrize("call", ["fa_plan_stats", "fa_plan_items"])
def test_work_list_without_room(call):
    out = subprocess.run([sys.executable, "-c", CODE.format(call=call)], capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=ROOT))
    assert out.returncode == 0, out.stderr[-500:]
    assert out.stdout.split() == ["FA_ERR_ALLOC", str(2 * 128 * 129 // 2)]
