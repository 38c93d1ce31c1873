"""Writes fa_tmem_asm.h: tcgen05.ld / tcgen05.st wrappers with long register lists.

Each load wrapper issues its tcgen05.ld instructions and the tcgen05.wait::ld in
ONE asm statement, so the compiler cannot touch the destination registers
before the tensor-memory data has landed. Run: python gen_tmem_asm.py
"""
import os

HERE = os.path.dirname(os.path.abspath(__file__))


def ld_fn(name, nchunks):
    n = 32 * nchunks
    regs = ", ".join(f"%{i}" for i in range(n))
    lines = []
    for c in range(nchunks):
        rl = ", ".join(f"%{c * 32 + i}" for i in range(32))
        lines.append(f'      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {{{rl}}}, [%{n + c}];\\n"')
    lines.append('      "tcgen05.wait::ld.sync.aligned;\\n"')
    outs = ", ".join(f'"=r"(r[{i}])' for i in range(n))
    ins = ", ".join(f'"r"(taddr + {32 * c}u)' for c in range(nchunks))
    del regs
    return (f"// {n} consecutive 32-bit TMEM columns of this thread's lane, then wait::ld.\n"
            f"__device__ __forceinline__ void {name}(uint32_t taddr, uint32_t (&r)[{n}]) {{\n"
            f"  asm volatile(\n" + "\n".join(lines) + "\n"
            f"      : {outs}\n"
            f"      : {ins}\n"
            f"      : \"memory\");\n}}\n")


def st_fn(n):
    rl = ", ".join(f"%{i + 1}" for i in range(n))
    ins = ", ".join(f'"r"(r[{i}])' for i in range(n))
    return (f"// {n} consecutive 32-bit TMEM columns of this thread's lane (no wait).\n"
            f"__device__ __forceinline__ void tmem_st{n}(uint32_t taddr, const uint32_t (&r)[{n}]) {{\n"
            "  asm volatile(\n"
            f'      "tcgen05.st.sync.aligned.32x32b.x{n}.b32 [%0], {{{rl}}};\\n"\n'
            f'      :\n      : "r"(taddr), {ins}\n'
            '      : "memory");\n}\n')


def main():
    out = ["// Generated by gen_tmem_asm.py; do not edit by hand.",
           "// tcgen05 32x32b shape: warp w reaches TMEM lanes 32*(w%4) .. 32*(w%4)+31,",
           "// thread t of the warp reads/writes lane 32*(w%4)+t.",
           "#pragma once", "#include <stdint.h>", "", "namespace fa {", "namespace dev {", ""]
    out.append(ld_fn("tmem_ld32_wait", 1))
    out.append(ld_fn("tmem_ld64_wait", 2))
    out.append(ld_fn("tmem_ld128_wait", 4))
    out.append(st_fn(8))
    out.append(st_fn(16))
    out.append(st_fn(32))
    out += ["}  // namespace dev", "}  // namespace fa", ""]
    with open(os.path.join(HERE, "fa_tmem_asm.h"), "w") as f:
        f.write("\n".join(out))


if __name__ == "__main__":
    main()
