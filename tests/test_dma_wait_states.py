"""The loads from memory to LDS that are written as assembly, as the compiler places them
(compiled for gfx950, nothing is run).  The compiler does not look into such a load, so what
the hardware asks around it has to be there by construction: five wait states between a vector
instruction that writes a scalar register and a vector memory instruction that reads it, and M0
set again before another instruction that reads it."""
import re
import subprocess

import pytest

from w4a16_grouped_expert_amd import _build

WAIT_STATES = 5

TILE_PRODUCT = """
#include "tile_product.hpp"
using namespace moe;
// the resource's words are lanes' values until right before the load
__global__ void k_resource(const char* const* p, uint32_t* out) {
  __shared__ __attribute__((aligned(1024))) char s[8192];
  const uint32_t lds = (uint32_t)(uintptr_t)s;
  const int lane = threadIdx.x;
  dma16(resource(p[lane], 4096u), 16u * lane, lds);
  stage_barrier<0>();
  out[lane] = *(const MOE_LDS uint32_t*)(uintptr_t)(lds + 4 * lane);
}
// the compiler's own loads to LDS in front and behind, which read M0 too
__global__ void k_m0(const uint32_t* g, const char* p, uint32_t* out) {
  __shared__ __attribute__((aligned(1024))) char s[8192];
  const uint32_t lds = (uint32_t)(uintptr_t)s;
  const int lane = threadIdx.x;
  __builtin_amdgcn_global_load_lds((const MOE_GLOBAL uint32_t*)(g + lane), (MOE_LDS uint32_t*)s, 4, 0, 0);
  dma16(resource(p, 4096u), 16u * lane, lds + 1024);
  __builtin_amdgcn_global_load_lds((const MOE_GLOBAL uint32_t*)(g + 64 + lane), (MOE_LDS uint32_t*)s, 4, 256, 0);
  stage_barrier<0>();
  out[lane] = *(const MOE_LDS uint32_t*)(uintptr_t)(lds + 4 * lane);
}
"""

PREFILL = r"""
#include "ffn_prefill.hip"
using namespace moe;
template <typename F>
__device__ void one_load(const char* const* p, uint32_t* out, F&& load) {
  __shared__ __attribute__((aligned(1024))) char s[8192];
  const uint32_t lds = lds_addr(s);
  const int lane = threadIdx.x;
  load(raw_rsrc(p[lane]), lane, lds);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  out[lane] = reinterpret_cast<volatile uint32_t*>(s)[lane];
}
__global__ void k_resource16(const char* const* p, uint32_t* out) {
  one_load(p, out, [](i32x4_t r, int lane, uint32_t lds) { buf_dma16(r, 16u * lane, 0, lds); });
}
__global__ void k_resource4(const char* const* p, uint32_t* out) {
  one_load(p, out, [](i32x4_t r, int lane, uint32_t lds) { buf_dma4(r, 4u * lane, 0, lds); });
}
"""


def instructions(source, tmp_path):
    """(mnemonic, operands) of each instruction, by kernel."""
    try:
        hipcc = _build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    src, asm = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(source)
    r = subprocess.run([hipcc, *_build.COMMON_FLAGS, "-w", "--cuda-device-only", "-S", str(src), "-o", str(asm)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    out, body = {}, []
    for line in asm.read_text().splitlines():
        text = line.split(";")[0].strip()
        label = re.match(r"(_Z\w+):", text)
        if label:
            body = out.setdefault(label[1], [])
        elif text and not text.startswith(".") and not text.endswith(":"):
            op, _, rest = text.partition(" ")
            body.append((op, [a.strip().split()[0] for a in re.split(r",\s*(?![^\[]*\])", rest) if a.strip()], text))
    return out


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]|s(\d+)", operand)
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def wait_states(body, at):
    """Between the last vector instruction that writes a scalar operand of body[at] and body[at]."""
    read = set().union(*[scalars(a) for a in body[at][1]])
    states = 0
    for op, operands, _ in reversed(body[:at]):
        if op.startswith("v_") and operands and scalars(operands[0]) & read:
            return states
        states += int(operands[0]) + 1 if op == "s_nop" else 1
    return None


def loads_to_lds(body):
    return [i for i, (op, _, text) in enumerate(body) if op.startswith(("buffer_load", "global_load")) and "lds" in text]


def kernel(found, name):
    return next(body for label, body in found.items() if name in label)


@pytest.mark.parametrize("source,name", [(TILE_PRODUCT, "k_resource"), (PREFILL, "k_resource16"),
                                         (PREFILL, "k_resource4")], ids=["tile_product", "prefill 16", "prefill 4"])
def test_wait_states_in_front_of_a_resource(source, name, tmp_path):
    body = kernel(instructions(source, tmp_path), name)
    loads = loads_to_lds(body)
    assert len(loads) == 1
    states = wait_states(body, loads[0])
    assert states is not None and states >= WAIT_STATES, body


def test_m0_is_set_again(tmp_path):
    """(The compiler keeps M0 between its own two loads where it sees nothing else write it.)"""
    body = kernel(instructions(TILE_PRODUCT, tmp_path), "k_m0")
    loads = loads_to_lds(body)
    assert len(loads) == 3
    for before, load in zip(loads, loads[1:]):
        assert any(operands[:1] == ["m0"] for _, operands, _ in body[before + 1:load]), body
