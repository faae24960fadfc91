// Host program: the rows that the gated scan's kernels are given, from the code
// that gives them.  A row that is read in pairs of channels has to lie on a
// pair's boundary in shared memory for every token of a warp, those that do not
// exist among them.  Prints what does not; compiled and run by
// test_gated_rows_cpu.py.
#include <cstdio>

#include "ssd_gated.cuh"

using namespace ssd;

static int bad = 0;

template <typename T>
static void check(const char *name, const Rows<const T> &r, const ssd_gated_shape_t &s, Align align) {
    if (align != kPairs) return;
    for (int b = 0; b < (int)s.batch; ++b) {
        const uint64_t first = reinterpret_cast<uintptr_t>(r.p) + (uint64_t)(b * r.bs) * sizeof(T);
        for (int t = 0; t < 32; ++t)
            if ((first + (uint64_t)t * (uint64_t)(int64_t)r.rs * sizeof(T)) % (2 * sizeof(T))) {
                std::printf("%s of %d bytes, batch %d, seqlen %d, strides %lld %d: token %d of row %d is off\n", name, (int)sizeof(T),
                            (int)s.batch, (int)s.seqlen, (long long)r.bs, r.rs, t, b);
                ++bad;
                return;
            }
    }
}

template <typename T>
static int sweep(ssd_dtype_t dtype) {
    int pairs = 0;
    char *base = reinterpret_cast<char *>(uintptr_t(1) << 20);
    for (int64_t batch : {1, 2, 3})
        for (int64_t L : {1, 2, 33})
            for (int64_t ch : {2, 66, 1002})
                for (int64_t rs : {0, 66, 67, 1003, 1006, 4001})
                    for (int64_t bs : {0, 335, 4012, 4013})
                        for (int at : {0, 2, 5})
                            for (int which = 0; which < 5; ++which) {  // the operand that is so; 4: an i that is not there
                                ssd_gated_shape_t s{batch, L, ch, 8.f, dtype};
                                const ssd_rows_t plain{base, L * ch, ch}, odd{base + at * sizeof(T), bs, rs};
                                ssd_gated_inputs_t in{plain, plain, plain, plain, nullptr, nullptr};
                                (which == 0 ? in.x : which == 1 ? in.r : which == 2 ? in.z : in.i) = odd;
                                if (which == 4) in.i.data = nullptr;
                                const Align align = gated_align(&s, &in);
                                pairs += align == kPairs;
                                const GatedArgs<T> a = gated_args<T>(&s, &in, batch);
                                check("x", a.x, s, align), check("r", a.r, s, align), check("z", a.z, s, align), check("i", a.i, s, align);
                                if (rows_pairs(odd, sizeof(T), batch, L)) check("another operand", gated_rows<const T>(&s, odd), s, align);
                            }
    return pairs;
}

int main() {
    const int pairs = sweep<bf16>(SSD_DTYPE_BF16) + sweep<float>(SSD_DTYPE_F32);
    std::printf("%d calls in pairs, %d operands off\n", pairs, bad);
    return bad || pairs == 0;
}
