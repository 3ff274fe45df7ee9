"""The wait between a matrix instruction and the first read of its result (csrc/weight_stream.h: settle, settle_all), on
the compiler's intermediate code: a value that is stored has to come from an instruction after the wait, so that no
pass can move the read in front of it.  Compiled for gfx950 on the CPU; nothing runs."""
import re
import subprocess

import pytest

from combine_expert_histogram_amd import build

PROBE = """
#include "weight_stream.h"
using namespace moe;
extern "C" __global__ void probe_settle(f32x4* p) {
    f32x4 d[5];
    for (int i = 0; i < 5; ++i) d[i] = p[i];
    settle(d);
    for (int i = 0; i < 5; ++i) p[8 + i] = d[i];
}
extern "C" __global__ void probe_settle_all(f32x4* p) {
    f32x4 d[3][2];
    for (int i = 0; i < 6; ++i) d[i / 2][i % 2] = p[i];
    settle_all(d);
    for (int i = 0; i < 6; ++i) p[8 + i] = d[i / 2][i % 2];
}
"""


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    where = tmp_path_factory.mktemp("probe")
    (where / "probe.hip").write_text(PROBE)
    flags = [f for f in build.flags() if f not in ("-fPIC", "-shared")]
    cmd = [build.hipcc(), *flags, "--cuda-device-only", "-S", "-emit-llvm", str(where / "probe.hip"), "-o",
           str(where / "probe.ll")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return (where / "probe.ll").read_text()


@pytest.mark.parametrize("name,tiles", [("probe_settle", 5), ("probe_settle_all", 6)])
def test_every_tile_is_read_after_the_wait(listing, name, tiles):
    body = re.search(r"define [^\n]*@%s\([^\n]*\n(.*?)\n}" % name, listing, re.S).group(1).split("\n")
    waits = [i for i, line in enumerate(body) if "s_nop 15" in line]
    assert len(waits) == 1
    defined = {}
    for i, line in enumerate(body):
        m = re.match(r"\s*(%[\w.]+) = (.*)", line)
        if m:
            defined[m[1]] = i, m[2]
    stored = [m[1] for m in (re.match(r"\s*store <4 x float> (%[\w.]+),", line) for line in body) if m]
    assert len(stored) == tiles
    for value in stored:
        at, what = defined[value]
        if "extractvalue" in what:                               # of the wait's own results
            at, what = defined[re.search(r"(%[\w.]+), \d+$", what)[1]]
        assert "asm sideeffect" in what and at >= waits[0], (value, what)
