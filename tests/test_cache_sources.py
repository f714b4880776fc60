"""Shared memory of the cache's attention, without a GPU: what a kernel lays out ends inside what its launch asks for, with
the 1023 bytes that the alignment of the first address may take to spare.  Checked by the compiler's front end alone: the
last assertion ends it, so that nothing is generated."""
import subprocess

import pytest

from self_attention_gb300.build import ARCH, CSRC, NVCC_FLAGS, nvcc

# end of the layout, sizes from the kernel's configuration C
LAYOUTS = [("FewCfg", d, nt, "C::RINGS + C::JOIN + kFewWarps * C::STAGES * 8 + 4") for d in (64, 128) for nt in (1, 2)]
LAYOUTS += [("UnitCfg", d, nt, "C::RINGS + (int)sizeof(C::Sum) + kUnitWarps * C::STAGES * 8 + 4") for d in (64, 128) for nt in (1, 2)]


@pytest.mark.parametrize("cfg,d,nt,end", LAYOUTS)
def test_layouts_end_inside_their_shared_memory(cfg, d, nt, end, tmp_path):
    source = tmp_path / "layout.cu"
    source.write_text(f"""#include "cache_attn.cu"
namespace attn {{
namespace {{
using C = {cfg}<{d}, {nt}>;
static_assert(({end}) + 1023 <= C::SMEM, "past the end");
static_assert(C::SMEM == 0, "the last line");
}}
}}
""")
    r = subprocess.run([nvcc(), *ARCH, *NVCC_FLAGS, "-c", str(source), "-o", str(tmp_path / "layout.o")],
                       capture_output=True, text=True)
    assert r.returncode != 0 and "the last line" in r.stderr, r.stderr
    assert r.stderr.count("error:") == 1 and "past the end" not in r.stderr, r.stderr
