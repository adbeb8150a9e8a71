"""Generated code of the experts' products (hipcc cross-compiles gfx950 here, no GPU needed).

Their loads go straight into LDS and run stages ahead of the products; the source waits for a stage
with counted waits.  A wait for every load in flight inside a loop of products, which the compiler adds
where it takes an LDS read for one of what a load in flight writes, gives the right results a third
slower; no parity test sees it."""
import re

import test_codegen_cpu as codegen


def _blocks(lines):
    """The basic blocks of a function: lists of instructions."""
    block = []
    for line in lines:
        if re.match(r"\.LBB\w+:", line):
            yield block
            block = []
        elif line and not line.startswith((";", ".")):
            block.append(line)
    yield block


def _kernels(asm):
    for name in re.findall(r"^\s*\.type\s+(_ZN3moe\w*k_experts\w+),@function", asm, re.M):
        i = asm.index("\n" + name + ":")
        yield name, [l.strip() for l in asm[i:asm.index(".Lfunc_end", i)].splitlines()]


def test_no_product_waits_for_the_loads_in_flight(tmp_path):
    asm, _ = codegen._device_asm(tmp_path, "experts.hip")
    kernels = list(_kernels(asm))
    assert len(kernels) == 4  # bf16 and e4m3, plain and gated
    for name, lines in kernels:
        products = [b for b in _blocks(lines) if any(l.startswith("v_mfma") for l in b)]
        # a loop for each kind of tile: 12, and 7 where a tile has whole blocks of 128 gated columns
        assert len(products) >= (7 if "ILb1ELb1E" in name else 12), name
        waits = [l for b in products for l in b if "vmcnt" in l]
        assert not waits, (name, waits)


def test_tiles_are_loaded_straight_into_lds(tmp_path):
    asm, _ = codegen._device_asm(tmp_path, "experts.hip")
    for name, lines in _kernels(asm):
        assert any(l.startswith("global_load_lds_dwordx4") for l in lines), name
        assert not any(re.match(r"(global|flat|buffer)_load_dwordx4", l) for l in lines), name
        assert not any(l.startswith("v_pk_") and "f32" in l for l in lines), name
