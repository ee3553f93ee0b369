// The block table as the attention-side kernels read it (q8_kv4_internal.h),
// compiled for the host: every slot and page id a caller's arrays may hold,
// with marked entries around the table.  Prints nothing; the exit status is the
// number of the check that failed.
#include <cstdint>
#include <vector>

#include "q8_kv4_internal.h"

int main() {
    const int n_slots = 3, max_pages = 5, page_tokens = 64, around = 4096;
    const int32_t mark = 1 << 20;  // what lies beside the table
    std::vector<int32_t> memory(2 * around + n_slots * max_pages, mark);
    for (int i = 0; i < n_slots * max_pages; ++i) memory[around + i] = i;
    q8::KvView c = {};
    c.table = memory.data() + around;
    c.n_pages = n_slots * max_pages - 1;  // the last entry names no page
    c.n_slots = n_slots;
    c.max_pages = max_pages;
    c.page_tokens = page_tokens;
    const int32_t ends[] = {INT32_MIN, INT32_MIN + 1, -1000000, -64, -2, -1, 0, 1, 2, 3, 4, 5, 6, 15, 16,
                            99, 319, 320, 321, 1000000, 1 << 30, INT32_MAX - 64, INT32_MAX - 1, INT32_MAX};
    for (int32_t s : ends)
        for (int32_t i : ends) {
            const bool in = s >= 0 && s < n_slots && i >= 0 && i < max_pages;
            if (q8::table_entry(c, s, i) != (in ? s * max_pages + i : -1)) return 1;
        }
    for (int32_t s : ends)
        for (int32_t p : ends) {
            const bool in = s >= 0 && s < n_slots && p >= 0 && p < max_pages * page_tokens;
            const int64_t page = in ? s * max_pages + p / page_tokens : -1;
            if (q8::kv_page(c, s, p) != (page < c.n_pages ? page : -1)) return 2;
        }
    // the largest table that the entry points take: the index passes 31 bits
    // nowhere in 64
    c.n_slots = INT32_MAX;
    c.max_pages = 1;
    if (q8::table_entry(c, -1, 0) != -1 || q8::table_entry(c, INT32_MAX, 0) != -1 ||
        q8::table_entry(c, 0, 1) != -1)
        return 3;
    return 0;
}
